// Softmax cross entropy of a linear classifier, without its logits.  For the rows
// r of x [R, I] with a class t = target[r] in [0, V), the others are left out,
// and a class's row w_v of w [V, I]:
//
//   l_rv = x_r.w_v      loss_r = log sum_v exp(l_rv) - l_rt
//   p_rv = exp(l_rv) / sum_v exp(l_rv)      d_rv = g_r (p_rv - [v = t])
//   dx_r = sum_v d_rv w_v                   dw_v = sum_r d_rv x_r
//
// Forward: the tiles of x w^T on the matrix cores (tile_product.h); each keeps
// the maximum and sum of its rows and the logit of their class, and a second
// kernel joins the tiles of a row.  Nothing of the size of the logits is written.
//
// Backward, in pieces of the classes that fit kPieceBytes: the tiles of the
// piece's logits once more, turned into d where they stand in the registers and
// stored in the rows' type; then the piece's dw, whole, and its part of dx, added
// up in fp32 over the pieces.  One product more than with the logits kept, at
// 2 I operations an element against a write and two reads of it.
//
// d is rounded to the rows' type because the matrix cores take it so; it is at
// most 1 in size there: the gradient's power of two is taken out and put back
// behind the sums, and fp16 holds d times 2^12 more, so that probabilities down to
// 2^-26 keep eleven bits.  One power of two for all rows, the largest row's: dw adds
// them up.  Where each row has a gradient of its own, what counts in fp16 is p times
// the row's share of the largest (256 rows of 64, dx of rows at 2^-16 of the largest 2.4e-4
// off, as rounding alone; at 2^-18 2.8e-4 with 4,000 classes and 2.7e-3 with 65,536, at
// 2^-24 0.02 and 0.12).  Sums are fp32.
//
// The rows with a class are listed on the device first.  The logits' tiles gather
// their rows by the list and dx is scattered by it, so rows without one cost
// nothing and what stands in them reaches nothing; dw's rows are packed for it
// when some are left out.
//
// Bound by the matrix cores; medians of the kernels alone under the profiler,
// 7,800 rows with a class x 2048, 65,536 classes, bf16: statistics 2,025 us (1.03
// PFLOP/s, matrix cores 57% busy), d 2,237 in two pieces (49%), dx 1,778 (62%), dw
// 1,662 (69%), against 1.21 PFLOP/s of a large library product; a tile of the
// logits sums over 2,048 elements, too few to cover its start and its exponentials.
// 64 rows x 2048, 32,768 classes: 26 us, w's 134 MB at 5.2 TB/s.  150,000 rows with a
// class of 300,007 x 128, 47 classes, fp32: 36 + 38 us for the tiles' two passes, dx 41,
// dw 34, 49 for packing rows and clearing the others: eight passes over the rows.
#include "tile_product.h"

namespace gspmm {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

using Narrow = Shape<64, 64, 2, 2>;
using Flat = Shape<64, 128, 1, 4>;

// ---- the rows with a class ----

constexpr int kListThreads = 256, kListRows = 2048;

__device__ inline bool has_class(const LossArgs &a, int64_t r) {
    const int64_t t = a.target[r];
    return t >= 0 && t < a.V;
}

// Inclusive sum over the block; *all: of the whole block.
__device__ inline int block_inclusive(int v, int *all) {
    __shared__ int waves[kListThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int up = __shfl_up(v, o, kWave);
        if (lane >= o) v += up;
    }
    __syncthreads();
    if (lane == kWave - 1) waves[wave] = v;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kListThreads / kWave; ++i) {
        if (i < wave) v += waves[i];
        sum += waves[i];
    }
    *all = sum;
    return v;
}

__global__ __launch_bounds__(kListThreads) void loss_count_kernel(LossArgs a) {
    const int64_t first = (int64_t)blockIdx.x * kListRows;
    int n = 0, all;
    for (int i = threadIdx.x; i < kListRows; i += kListThreads) n += first + i < a.R && has_class(a, first + i);
    block_inclusive(n, &all);
    if (threadIdx.x == 0) a.block_count[blockIdx.x] = all;
}

// A block's rows behind those of the blocks before it.
__global__ __launch_bounds__(kListThreads) void loss_list_kernel(LossArgs a, int blocks) {
    const int64_t first = (int64_t)blockIdx.x * kListRows;
    int before = 0, all, n = 0;
    for (int b = threadIdx.x; b < (int)blockIdx.x; b += kListThreads) before += a.block_count[b];
    block_inclusive(before, &before);
    constexpr int kPer = kListRows / kListThreads;
    bool in[kPer];
    const int64_t mine = first + (int64_t)threadIdx.x * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        in[i] = mine + i < a.R && has_class(a, mine + i);
        n += in[i];
    }
    int at = before + block_inclusive(n, &all) - n;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (in[i]) a.rows[at++] = (int)(mine + i);
        else if (a.per_row && mine + i < a.R) a.row_loss[mine + i] = 0.0f;
    }
    if (blockIdx.x == blocks - 1 && threadIdx.x == 0) *a.count = before + all;
}

// ---- tiles ----

struct TileAt {
    int64_t row, col;       // in tiles
};

// Tile number id of rows x cols tiles: an XCD takes a run of them, and within it
// 8 row tiles meet each column tile in turn, so that the tiles under way at one
// time share both operands in its L2.
constexpr int kGroupRows = 8;

__device__ inline TileAt tile_at(int64_t id, int64_t rows, int64_t cols) {
    const int64_t total = rows * cols, per = total / 8, extra = total % 8, x = id % 8;
    const int64_t at = x * per + (x < extra ? x : extra) + id / 8;
    const int64_t group = at / (kGroupRows * cols), in = at % (kGroupRows * cols);
    const int64_t high = min(int64_t(kGroupRows), rows - group * kGroupRows);
    return {group * kGroupRows + in % high, in / high};
}

__device__ inline int register_col(int e) { return 8 * (e >> 2) + 4 * ((threadIdx.x & (kWave - 1)) >> 5) + (e & 3); }

__device__ inline float other_half(float v) { return __shfl_xor(v, 32, kWave); }

// A class's column among the n from n0 on of a tile, -1 if it is another's.
__device__ inline int in_tile(int64_t t, int n0, int n) { return t >= n0 && t < n0 + n ? (int)t - n0 : -1; }

// What d's rows are multiplied with, and the sums with its inverse.
template <typename T>
constexpr float kHeld = __is_same(T, _Float16) ? 4096.0f : 1.0f;

__device__ inline float loss_unit(const LossArgs &a) {
    if (a.per_row) return *a.unit;
    const int64_t n = *a.count;
    return a.mean ? *a.dloss / (float)max(n, int64_t(1)) : *a.dloss;
}

// A tile of the logits of the classes [v0, v0 + N): its rows' statistics, or
// (BACKWARD) d.
template <typename T, typename S, bool DIRECT, bool BACKWARD>
__global__ __launch_bounds__(S::kThreads, 2) void loss_logits_kernel(LossArgs a, int64_t v0, int64_t N, int64_t total) {
    TILE_STAGES(lds, S::kStageBytes);
    const int64_t count = *a.count, row_tiles = (count + S::BM - 1) / S::BM, col_tiles = (N + S::BN - 1) / S::BN;
    const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
    const int wc = wave % S::WC, m0 = wave / S::WC * (S::MI * 32), n0 = wc * (S::NI * 32);
    for (int64_t id = blockIdx.x; id < min(total, row_tiles * col_tiles); id += gridDim.x) {
        const TileAt at = tile_at(id, row_tiles, col_tiles);
        const int64_t row = uniform(at.row * S::BM), col = uniform(at.col * S::BN);
        Operand<T> A, B;
        A.ptr = (const T *)a.x;
        A.ld = a.ld;
        A.outer = count - row;
        A.inner = a.ld;
        A.end = A.ptr + a.R * a.ld;
        A.rows = a.rows + row;
        B.ptr = (const T *)a.w + (v0 + col) * a.ld;
        B.ld = a.ld;
        B.outer = N - col;
        B.inner = a.ld;
        B.end = (const T *)a.w + a.V * a.ld;
        __syncthreads();
        Sums<S> sums = {};
        f32x16 (&acc)[S::MI][S::NI] = sums.at;
        tile_sums<T, S, true, true, DIRECT, true>(lds, A, B, a.ld, sums);
        const int left = (int)min(int64_t(S::BN), N - col);
        // columns behind the last class: in the last tile alone
        if (left < S::BN) {
#pragma unroll
            for (auto &line : acc)
#pragma unroll
                for (int j = 0; j < S::NI; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (n0 + j * 32 + register_col(e) >= left) line[j][e] = -INFINITY;
        }
        if constexpr (BACKWARD) {
#pragma unroll
            for (int i = 0; i < S::MI; ++i) {
                const int64_t r = min(row + m0 + i * 32 + (lane & 31), count - 1);
                const float top = a.stats[r], inverse = a.stats[a.R + r];
                const int t = in_tile(a.target[a.rows[r]] - v0 - col, n0, S::NI * 32);
                const float g = a.per_row ? a.dloss[a.rows[r]] / *a.unit * kHeld<T> : kHeld<T>;
                const float pg = inverse * g, from = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (auto &block : acc[i])
#pragma unroll
                    for (int e = 0; e < 16; ++e) block[e] = __builtin_amdgcn_exp2f((block[e] - from) * kLog2e) * pg;
                if (__any(t >= 0)) {
#pragma unroll
                    for (int j = 0; j < S::NI; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (j * 32 + register_col(e) == t) acc[i][j][e] -= g;
                }
            }
            tile_store<T, S>(lds, sums, (T *)a.d + row * a.ldd + col, a.ldd, count - row, a.ldd - col, false);
        } else {
            auto *joint = (__attribute__((address_space(3))) float *)lds.at[0];
#pragma unroll
            for (int i = 0; i < S::MI; ++i) {
                const int in = m0 + i * 32 + (lane & 31);
                const int64_t r = min(row + in, count - 1);
                const int t = in_tile(a.target[a.rows[r]] - v0 - col, n0, S::NI * 32);
                if (__any(t >= 0)) {
                    float picked = 0.0f;
                    bool mine = false;
#pragma unroll
                    for (int j = 0; j < S::NI; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (j * 32 + register_col(e) == t) {
                                picked = acc[i][j][e];
                                mine = true;
                            }
                    if (mine && row + in < count) a.picked[r] = picked;
                }
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int j = 0; j < S::NI; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, acc[i][j][e]);
                top = fmaxf(top, other_half(top));
                const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int j = 0; j < S::NI; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum += __builtin_amdgcn_exp2f((acc[i][j][e] - from) * kLog2e);
                sum += other_half(sum);
                if (lane < 32) {
                    joint[(in * S::WC + wc) * 2] = top;
                    joint[(in * S::WC + wc) * 2 + 1] = sum;
                }
            }
            __syncthreads();
            if (threadIdx.x < S::BM && row + threadIdx.x < count) {
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int c = 0; c < S::WC; ++c) top = fmaxf(top, joint[(threadIdx.x * S::WC + c) * 2]);
                const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int c = 0; c < S::WC; ++c)
                    sum += joint[(threadIdx.x * S::WC + c) * 2 + 1] *
                           __builtin_amdgcn_exp2f((joint[(threadIdx.x * S::WC + c) * 2] - from) * kLog2e);
                const int64_t to = at.col * a.R + row + threadIdx.x;
                a.tile_top[to] = top;
                a.tile_sum[to] = sum;
            }
        }
    }
}

// ---- the rows' losses ----

constexpr int kJoinThreads = 256, kJoinRows = 32;

// Rows of a block: 32, or 8 where a row has many tiles (256 tiles of 64 rows: 11 -> 5 us).
int join_rows(int tiles) { return tiles > 32 ? 8 : kJoinRows; }

// Joins the column tiles of ROWS rows, 256 / ROWS tiles at a time.
template <int ROWS>
__global__ __launch_bounds__(kJoinThreads) void loss_join_kernel(LossArgs a, int tiles) {
    constexpr int kGroups = kJoinThreads / ROWS;
    __shared__ float tops[kGroups][ROWS], sums[kGroups][ROWS];
    const int64_t count = *a.count;
    const int in = threadIdx.x % ROWS, group = threadIdx.x / ROWS;
    for (int64_t block = blockIdx.x; block * ROWS < a.R; block += gridDim.x) {
        const int64_t r = block * ROWS + in;
        float top = -INFINITY, sum = 0.0f;
        if (r < count) {
#pragma unroll 4
            for (int t = group; t < tiles; t += kGroups) {
                const float tile_top = a.tile_top[t * a.R + r], tile_sum = a.tile_sum[t * a.R + r];
                const float next = fmaxf(top, tile_top), from = next == -INFINITY ? 0.0f : next;
                sum = sum * __builtin_amdgcn_exp2f((top - from) * kLog2e) +
                      tile_sum * __builtin_amdgcn_exp2f((tile_top - from) * kLog2e);
                top = next;
            }
        }
        __syncthreads();
        tops[group][in] = top;
        sums[group][in] = sum;
        __syncthreads();
        if (threadIdx.x < kWave) {
            float loss = 0.0f;
            if (threadIdx.x < ROWS && r < count) {
                top = -INFINITY;
                sum = 0.0f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) top = fmaxf(top, tops[g][in]);
                const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    sum += sums[g][in] * __builtin_amdgcn_exp2f((tops[g][in] - from) * kLog2e);
                loss = (top - a.picked[r]) + logf(sum);
                a.stats[r] = top;
                a.stats[a.R + r] = 1.0f / sum;
                if (a.per_row) a.row_loss[a.rows[r]] = loss;
            }
            if (a.block_loss) {
#pragma unroll
                for (int o = ROWS / 2; o > 0; o >>= 1) loss += __shfl_xor(loss, o, kWave);
                if (threadIdx.x == 0) a.block_loss[block] = loss;
            }
        }
    }
}

constexpr int kTotalThreads = 1024;

// v of the whole block, by `join`, in a fixed order.
template <typename F>
__device__ inline float block_all(float v, F join) {
    __shared__ float waves[kTotalThreads / kWave];
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v = join(v, __shfl_xor(v, o, kWave));
    if ((threadIdx.x & (kWave - 1)) == 0) waves[threadIdx.x / kWave] = v;
    __syncthreads();
    v = waves[0];
#pragma unroll
    for (int i = 1; i < kTotalThreads / kWave; ++i) v = join(v, waves[i]);
    return v;
}

__global__ __launch_bounds__(kTotalThreads) void loss_total_kernel(LossArgs a, int64_t blocks) {
    float sum = 0.0f;
    for (int64_t i = threadIdx.x; i < blocks; i += kTotalThreads) sum += a.block_loss[i];
    sum = block_all(sum, [](float x, float y) { return x + y; });
    if (threadIdx.x == 0) *a.loss = a.mean ? sum / (float)max(*a.count, int64_t(1)) : sum;
}

// ---- backward ----

// The power of two above the largest gradient of a row (1 where all are zero): the
// blocks' largest, and theirs where there is more than one block.
constexpr int kUnitRows = 16384;
constexpr int64_t kUnitBlocks = 1024;

__device__ inline void store_unit(const LossArgs &a, float most) {
    *a.unit = most > 0.0f ? ldexpf(1.0f, min(max(ilogbf(most) + 1, -120), 120)) : 1.0f;
}

__global__ __launch_bounds__(kTotalThreads) void loss_unit_kernel(LossArgs a) {
    const int64_t count = *a.count;
    float most = 0.0f;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.x * kTotalThreads + threadIdx.x; r < count;
         r += (int64_t)gridDim.x * kTotalThreads) {
        const float g = fabsf(a.dloss[a.rows[r]]);
        most = g <= 3.0e38f ? fmaxf(most, g) : most;     // infinities and NaN: theirs alone
    }
    most = block_all(most, [](float x, float y) { return fmaxf(x, y); });
    if (threadIdx.x) return;
    if (gridDim.x > 1) a.unit[1 + blockIdx.x] = most;
    else store_unit(a, most);
}

__global__ __launch_bounds__(kTotalThreads) void loss_unit_join_kernel(LossArgs a, int blocks) {
    const float most = block_all((int)threadIdx.x < blocks ? a.unit[1 + threadIdx.x] : 0.0f,
                                 [](float x, float y) { return fmaxf(x, y); });
    if (threadIdx.x == 0) store_unit(a, most);
}

// x's listed rows next to each other, where some are left out.
constexpr int kPackThreads = 256;

template <typename T>
__global__ __launch_bounds__(kPackThreads) void loss_pack_kernel(LossArgs a) {
    const int64_t count = *a.count, packs = (a.ld + kPack<T> - 1) / kPack<T>;
    if (count == a.R) return;
    for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < count * packs;
         i += (int64_t)gridDim.x * kPackThreads) {
        const int64_t r = i / packs, c = i % packs * kPack<T>;
        store_pack((T *)a.packed + r * a.ld + c, load_pack((const T *)a.x + a.rows[r] * a.ld + c, a.ld - c), a.ld - c);
    }
}

// Rows of I elements moved ld apart, zeros behind each; `listed`: those that have
// a class alone.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void loss_pad_kernel(LossArgs a, const T *from, T *to, int64_t rows,
                                                                int64_t I, int64_t ld, bool listed) {
    const int64_t packs = ld / kPack<T>;
    for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < rows * packs;
         i += (int64_t)gridDim.x * kPackThreads) {
        const int64_t r = i / packs, c = i % packs * kPack<T>;
        if (listed && !has_class(a, r)) continue;
        store_pack(to + r * ld + c, load_pack(from + r * I + c, I - c), kPack<T>);
    }
}

// dx of the rows that are left out, and (pieces) of the others from its fp32 sums.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void loss_rest_kernel(LossArgs a, bool summed) {
    const int64_t packs = (a.I + kPack<T> - 1) / kPack<T>, count = *a.count, zeros = count == a.R ? 0 : a.R;
    const float f = summed ? loss_unit(a) / kHeld<T> : 0.0f;
    for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < ((summed ? count : 0) + zeros) * packs;
         i += (int64_t)gridDim.x * kPackThreads) {
        const int64_t r = i / packs, c = i % packs * kPack<T>;
        Pack<T> v;
        int64_t to = r;
        if (r >= zeros) {
            to = a.rows[r - zeros];
            float sum[kPack<T>] = {};
            for (int64_t p = 0; p < a.dx_parts; ++p) {
                const float *from = a.dx_sum + (p * a.R + r - zeros) * a.I + c;
#pragma unroll
                for (int q = 0; q < kPack<T>; q += 4) {
                    const Pack<float> part = load_pack(from + q, a.I - c - q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[q + e] += part.v[e];
                }
            }
#pragma unroll
            for (int e = 0; e < kPack<T>; ++e) v.v[e] = (T)(sum[e] * f);
        } else {
            if (has_class(a, r)) continue;
#pragma unroll
            for (int e = 0; e < kPack<T>; ++e) v.v[e] = (T)0.0f;
        }
        store_pack((T *)a.dx + to * a.I + c, v, a.I - c);
    }
}

// A tile's sums over K: fp32 rows in runs of kRun that are added up at their ends,
// since one chain over all of K rounds to the size of its largest term at each step
// (6,000 rows of 1024, 8,000 classes: dx 1.6e-6 off and 3,051 us in one chain, 1.1e-6
// and 3,072 us in runs of 4,096, 8e-7 and 3,072 us of 2,048; sums of like terms, 65,536
// rows through registers: 9.8e-4 off in one chain, 3.2e-5 in runs).  16-bit results are
// rounded far above that, and dx in small tiles (rows by rows) sums over 64 classes at most.
constexpr int64_t kRun = 2048;

template <typename T, typename S, bool A_ROWS, bool DIRECT>
__device__ inline void long_sums(const Stages &lds, const Operand<T> &a, const Operand<T> &b, int64_t K,
                                 Sums<S> &sums) {
    if constexpr (sizeof(T) == 2 || (A_ROWS && S::BM == Narrow::BM)) {
        tile_sums<T, S, A_ROWS, false, DIRECT>(lds, a, b, K, sums);
    } else {
        for (int64_t k = 0; k < K; k += kRun) {
            const int64_t n = min(kRun, K - k);
            Operand<T> A = a, B = b;
            A.ptr += A_ROWS ? k : k * a.ld;
            (A_ROWS ? A.inner : A.outer) = n;
            B.ptr += k * b.ld;
            B.outer = min(n, b.outer - k);
            Sums<S> run = {};
            tile_sums<T, S, A_ROWS, false, DIRECT>(lds, A, B, n, run);
#pragma unroll
            for (int i = 0; i < S::MI; ++i)
#pragma unroll
                for (int j = 0; j < S::NI; ++j) sums.at[i][j] += run.at[i][j];
        }
    }
}

// A tile of dx = d w over a part of a piece's classes: ADD is -1 where it is the
// whole of dx, 0 and 1 for the first and the other pieces of the fp32 sums.
template <typename T, typename S, bool DIRECT, int ADD>
__global__ __launch_bounds__(S::kThreads, 2) void loss_dx_kernel(LossArgs a, int64_t first, int64_t classes,
                                                                 int64_t total) {
    TILE_STAGES(lds, S::kStageBytes);
    const int64_t count = *a.count, row_tiles = (count + S::BM - 1) / S::BM, col_tiles = (a.I + S::BN - 1) / S::BN;
    for (int64_t id = blockIdx.x; id < min(total, row_tiles * col_tiles * a.dx_parts); id += gridDim.x) {
        const int64_t part = ADD < 0 ? 0 : id / (row_tiles * col_tiles), skip = part * a.dx_part;
        const int64_t v0 = first + skip, N = ADD < 0 ? classes : max(int64_t(0), min(a.dx_part, classes - skip));
        // behind the last class d holds zeros up to whole packs
        const int64_t K = (N + kPack<T> - 1) / kPack<T> * kPack<T>;
        const TileAt at = tile_at(id - part * row_tiles * col_tiles, row_tiles, col_tiles);
        const int64_t row = uniform(at.row * S::BM), col = uniform(at.col * S::BN);
        Operand<T> A, B;
        A.ptr = (const T *)a.d + row * a.ldd + skip;
        A.ld = a.ldd;
        A.outer = count - row;
        A.inner = K;
        A.end = (const T *)a.d + a.R * a.ldd;
        B.ptr = (const T *)a.w + v0 * a.ld + col;
        B.ld = a.ld;
        B.outer = N;
        B.inner = a.I - col;
        B.end = (const T *)a.w + a.V * a.ld;
        __syncthreads();
        Sums<S> sums = {};
        f32x16 (&acc)[S::MI][S::NI] = sums.at;
        long_sums<T, S, true, DIRECT>(lds, A, B, K, sums);
        if constexpr (ADD < 0) {
            const float f = loss_unit(a) / kHeld<T>;
#pragma unroll
            for (auto &line : acc)
#pragma unroll
                for (auto &v : line) v *= f;
            tile_store<T, S, true>(lds, sums, (T *)a.dx + col, a.I, A.outer, B.inner, false, a.rows + row);
        } else {
            tile_store_fp32<S, ADD == 1>(sums, a.dx_sum + (part * a.R + row) * a.I + col, a.I, A.outer, B.inner);
        }
    }
}

// A tile of dw = d^T x of a piece's classes, over all listed rows or (chunk > 0)
// those of a chunk, as fp32 partial sums.
template <typename T, typename S, bool DIRECT>
__global__ __launch_bounds__(S::kThreads, 2) void loss_dw_kernel(LossArgs a, int64_t v0, int64_t N, int64_t chunk,
                                                                 int64_t total) {
    TILE_STAGES(lds, S::kStageBytes);
    const int64_t count = *a.count, row_tiles = (N + S::BM - 1) / S::BM, col_tiles = (a.I + S::BN - 1) / S::BN;
    const T *x = (const T *)(count == a.R ? a.x : a.packed);
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int64_t part = chunk ? id / (row_tiles * col_tiles) : 0;
        const TileAt at = tile_at(id - part * row_tiles * col_tiles, row_tiles, col_tiles);
        const int64_t row = uniform(at.row * S::BM), col = uniform(at.col * S::BN);
        const int64_t from = uniform(min(count, part * chunk)), n = chunk ? min(chunk, count - from) : count;
        Operand<T> A, B;
        A.ptr = (const T *)a.d + from * a.ldd + row;
        A.ld = a.ldd;
        A.outer = n;
        A.inner = N - row;
        A.end = (const T *)a.d + a.R * a.ldd;
        B.ptr = x + from * a.ld + col;
        B.ld = a.ld;
        B.outer = n;
        B.inner = a.I - col;
        B.end = x + a.R * a.ld;
        __syncthreads();
        Sums<S> sums = {};
        f32x16 (&acc)[S::MI][S::NI] = sums.at;
        long_sums<T, S, false, DIRECT>(lds, A, B, n, sums);
        if (chunk) {
            tile_store_fp32<S, false>(sums, a.dw_partial + (part * N + row) * a.I + col, a.I, A.inner, B.inner);
            continue;
        }
        const float f = loss_unit(a) / kHeld<T>;
#pragma unroll
        for (auto &line : acc)
#pragma unroll
            for (auto &v : line) v *= f;
        T *dw = (T *)a.dw + (v0 + row) * a.I + col;
        // a stage of flat tiles does not hold 32 of their fp32 rows
        if constexpr (sizeof(T) == 4 && S::BM == Flat::BM) tile_store_fp32<S, false>(sums, dw, a.I, A.inner, B.inner);
        else tile_store<T, S>(lds, sums, dw, a.I, A.inner, B.inner, false);
    }
}

// Adds dw's partial sums: a block takes 32 elements, eight runs of their chunks at a
// time, and adds the runs in their order.
constexpr int kFoldRuns = 8, kFoldElements = kPackThreads / kFoldRuns;

template <typename T>
__global__ __launch_bounds__(kPackThreads) void loss_fold_kernel(LossArgs a, int64_t v0, int64_t n, int64_t chunk) {
    __shared__ float runs[kFoldRuns][kFoldElements];
    const int64_t parts = (*a.count + chunk - 1) / chunk, per = (parts + kFoldRuns - 1) / kFoldRuns;
    const float f = loss_unit(a) / kHeld<T>;
    const int in = threadIdx.x % kFoldElements, run = threadIdx.x / kFoldElements;
    for (int64_t i0 = (int64_t)blockIdx.x * kFoldElements; i0 < n; i0 += (int64_t)gridDim.x * kFoldElements) {
        const int64_t i = i0 + in;
        float t = 0.0f;
        if (i < n) {
#pragma unroll 8
            for (int64_t p = run * per; p < min(parts, (run + 1) * per); ++p) t += a.dw_partial[p * n + i];
        }
        __syncthreads();
        runs[run][in] = t;
        __syncthreads();
        if (run == 0 && i < n) {
            t = 0.0f;
#pragma unroll
            for (int r = 0; r < kFoldRuns; ++r) t += runs[r][in];
            ((T *)a.dw)[v0 * a.I + i] = (T)(t * f);
        }
    }
}

// ---- the launches ----

constexpr int64_t kMaxBlocks = 1 << 20;
constexpr int64_t kUnits = 256;                      // compute units

// d of a piece of the classes: workspace, and what the next two products read.
constexpr int64_t kPieceBytes = int64_t(512) << 20;

int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

int64_t whole(int64_t n, int64_t of) { return (n + of - 1) / of * of; }

// Classes of a piece, and the elements of a row of d.
int64_t piece_of(int64_t R, int64_t V, int size) {
    const int64_t fits = std::max<int64_t>(256, kPieceBytes / std::max<int64_t>(1, R * size) / 256 * 256);
    return std::min(fits, whole(V, 16));
}

// 256 x 256 tiles when there are enough of them to fill the chip; 64 x 64 where no
// more columns exist: more of them share a unit, and their rounds end closer
// together than 128 x 64 ones' (1,000,000 rows of 64, half with a class, 40 classes, fp32,
// 474 -> 470 us; dx in such tiles too, see dx_shape(), 418).
enum class Tiles { kLarge, kMedium, kNarrow };

Tiles tiles_for(int64_t rows, int64_t cols, int size, bool direct) {
    if (cols <= 64) return Tiles::kNarrow;
    if (direct && size == 2 && cols > 128 && tiles_of(rows, 256) * tiles_of(cols, 256) >= 2 * kUnits)
        return Tiles::kLarge;
    return Tiles::kMedium;
}

int tile_cols(Tiles t) { return t == Tiles::kLarge ? 256 : t == Tiles::kMedium ? 128 : 64; }

// The copy into LDS needs rows of whole 16-byte groups from a 16-byte address,
// and 32-bit offsets from the start of x.
bool direct_rows(const void *p, int64_t rows, int64_t width, int size) {
    return (uintptr_t)p % 16 == 0 && width * size % 16 == 0 && rows * width * size < (int64_t(1) << 31);
}

// dw: all rows at once where its tiles fill the chip twice or there are few rows,
// else chunks of them, about two tiles of work for each compute unit.
int64_t dw_chunk(int64_t R, int64_t N, int64_t I) {
    const int64_t tiles = tiles_of(N, N <= 64 ? 64 : 128) * tiles_of(I, 128);
    const int64_t want = std::max<int64_t>(1, 2 * kUnits / tiles);
    if (tiles >= 2 * kUnits || R <= 1024 || want == 1) return 0;
    return whole(std::max<int64_t>(256, (R + want - 1) / want), 32);
}

// dx: 256 x 256 tiles where a piece has enough classes for their start and end to
// weigh little, and parts of the classes side by side, added up afterwards, where
// the tiles do not fill the chip (parts of 1,024 classes at least; 5,003 x 1001, 49,999
// classes, fp16: 1,165 us whole in 128 x 128 tiles, 529 in three parts of 256 x 256).  Up
// to 64 classes: a few steps to a tile, small tiles.
struct DxShape {
    bool large, small;
    int64_t parts, part;
};

DxShape dx_shape(int64_t R, int64_t I, int64_t N, int size, bool direct) {
    DxShape d;
    d.large = direct && size == 2 && I > 128 && R > 128 && N >= 4096;
    d.small = N <= 64;
    const int tile = d.large ? 256 : d.small ? 64 : 128;
    const int64_t tiles = tiles_of(R, tile) * tiles_of(I, tile), want = d.large ? kUnits : 2 * kUnits;
    d.parts = std::max<int64_t>(1, std::min({(want + tiles / 2) / std::max<int64_t>(1, tiles), N / 1024, int64_t(64)}));
    d.part = whole(tiles_of(N, (int)d.parts), 64);
    return d;
}

template <typename T, typename S, bool DIRECT, bool BACKWARD>
hipError_t logits_launch(const LossArgs &a, int64_t v0, int64_t N, hipStream_t s) {
    const int64_t total = tiles_of(a.R, S::BM) * tiles_of(N, S::BN);
    loss_logits_kernel<T, S, DIRECT, BACKWARD>
        <<<(unsigned)std::min(total, kMaxBlocks), S::kThreads, 0, s>>>(a, v0, N, total);
    return hipGetLastError();
}

template <typename T, bool BACKWARD>
hipError_t logits(const LossArgs &a, int64_t v0, int64_t N, Tiles tiles, bool direct, hipStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (tiles == Tiles::kLarge) return logits_launch<T, Large, true, BACKWARD>(a, v0, N, s);
    if (tiles == Tiles::kNarrow)
        return direct ? logits_launch<T, Narrow, true, BACKWARD>(a, v0, N, s)
                      : logits_launch<T, Narrow, false, BACKWARD>(a, v0, N, s);
    return direct ? logits_launch<T, Medium, true, BACKWARD>(a, v0, N, s)
                  : logits_launch<T, Medium, false, BACKWARD>(a, v0, N, s);
}

template <typename T, typename S, bool DIRECT>
hipError_t dx_launch(const LossArgs &a, int64_t v0, int64_t N, int add, hipStream_t s) {
    const int64_t total = tiles_of(a.R, S::BM) * tiles_of(a.I, S::BN) * a.dx_parts;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    if (add < 0) loss_dx_kernel<T, S, DIRECT, -1><<<blocks, S::kThreads, 0, s>>>(a, v0, N, total);
    else if (add == 0) loss_dx_kernel<T, S, DIRECT, 0><<<blocks, S::kThreads, 0, s>>>(a, v0, N, total);
    else loss_dx_kernel<T, S, DIRECT, 1><<<blocks, S::kThreads, 0, s>>>(a, v0, N, total);
    return hipGetLastError();
}

template <typename T, typename S, bool DIRECT>
hipError_t dw_launch(const LossArgs &a, int64_t v0, int64_t N, int64_t chunk, hipStream_t s) {
    const int64_t total = tiles_of(N, S::BM) * tiles_of(a.I, S::BN) * (chunk ? tiles_of(a.R, (int)chunk) : 1);
    loss_dw_kernel<T, S, DIRECT><<<(unsigned)std::min(total, kMaxBlocks), S::kThreads, 0, s>>>(a, v0, N, chunk, total);
    return hipGetLastError();
}

// Rows off 16 bytes are moved to whole ones first where the products (R V) outweigh
// the copies (R + V) by kPadGain.  1001 elements, fp16, 50,000 classes, with gradients:
// 256 rows 420 us moved and 366 as they are, 512 567 and 555, 1,024 761 and 934; 50
// classes, 30,000 rows of 101 91 and 60.
constexpr int64_t kPadGain = 512;

int64_t padded_width(int64_t R, int64_t I, int64_t V, int size) {
    const int64_t ld = whole(I, 16 / size);
    const bool gains = R * V > kPadGain * (R + V);
    return ld != I && gains && R * ld * size < (int64_t(1) << 31) && 320 * ld * size < (int64_t(1) << 31) ? ld : I;
}

// Bytes of both moved arrays, x first.
int64_t padded_bytes(int64_t R, int64_t I, int64_t V, int size) {
    const int64_t ld = padded_width(R, I, V, size);
    return ld == I ? 0 : whole(R * ld * size, 256) + whole(V * ld * size, 256);
}

template <typename T>
hipError_t pad(LossArgs &a, hipStream_t s) {
    a.ld = padded_width(a.R, a.I, a.V, sizeof(T));
    if (a.ld == a.I) return hipSuccess;
    T *x = (T *)a.padded, *w = x + whole(a.R * a.ld * sizeof(T), 256) / sizeof(T);
    auto blocks = [&](int64_t rows) {
        return (unsigned)std::min(std::max<int64_t>(1, rows * a.ld / kPack<T> / kPackThreads), int64_t(1) << 14);
    };
    loss_pad_kernel<T><<<blocks(a.R), kPackThreads, 0, s>>>(a, (const T *)a.x, x, a.R, a.I, a.ld, true);
    loss_pad_kernel<T><<<blocks(a.V), kPackThreads, 0, s>>>(a, (const T *)a.w, w, a.V, a.I, a.ld, false);
    a.x = x;
    a.w = w;
    return hipGetLastError();
}

template <typename T>
hipError_t forward(LossArgs a, hipStream_t s) {
    const int64_t blocks = std::max<int64_t>(1, tiles_of(a.R, kListRows));
    if (blocks > 1) loss_count_kernel<<<(unsigned)blocks, kListThreads, 0, s>>>(a);
    loss_list_kernel<<<(unsigned)blocks, kListThreads, 0, s>>>(a, (int)blocks);
    if (const hipError_t e = hipGetLastError()) return e;
    if (const hipError_t e = pad<T>(a, s)) return e;
    const bool direct = direct_rows(a.x, a.R, a.ld, sizeof(T)) && direct_rows(a.w, 320, a.ld, sizeof(T));
    const Tiles tiles = tiles_for(a.R, a.V, sizeof(T), direct);
    const int cols = (int)tiles_of(a.V, tile_cols(tiles));
    const int64_t joins = tiles_of(a.R, join_rows(cols));
    if (a.R > 0) {
        if (const hipError_t e = logits<T, false>(a, 0, a.V, tiles, direct, s)) return e;
        const unsigned n = (unsigned)std::min(joins, kMaxBlocks);
        if (join_rows(cols) == 8) loss_join_kernel<8><<<n, kJoinThreads, 0, s>>>(a, cols);
        else loss_join_kernel<kJoinRows><<<n, kJoinThreads, 0, s>>>(a, cols);
    }
    if (a.block_loss) loss_total_kernel<<<1, kTotalThreads, 0, s>>>(a, joins);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(const LossArgs &args, hipStream_t s) {
    LossArgs a = args;
    const int size = sizeof(T);
    const int64_t piece = piece_of(a.R, a.V, size), pieces = tiles_of(a.V, (int)piece);
    a.ldd = piece;
    if (const hipError_t e = pad<T>(a, s)) return e;
    const bool direct = direct_rows(a.x, a.R, a.ld, size) && direct_rows(a.w, 320, a.ld, size) &&
                        direct_rows(nullptr, 320, a.ldd, size);
    if (a.per_row) {
        const int blocks = (int)std::max<int64_t>(1, std::min(kUnitBlocks, a.R / kUnitRows));
        loss_unit_kernel<<<(unsigned)blocks, kTotalThreads, 0, s>>>(a);
        if (blocks > 1) loss_unit_join_kernel<<<1, kTotalThreads, 0, s>>>(a, blocks);
    }
    const int64_t packs = a.R * tiles_of(a.ld, kPack<T>);
    const unsigned pack_blocks = (unsigned)std::min(std::max<int64_t>(1, packs / kPackThreads), int64_t(1) << 14);
    if (a.dw) loss_pack_kernel<T><<<pack_blocks, kPackThreads, 0, s>>>(a);
    if (const hipError_t e = hipGetLastError()) return e;
    // the first piece is the largest: its parts serve all
    const DxShape dx = dx_shape(a.R, a.I, std::min(piece, a.V), size, direct);
    a.dx_parts = dx.parts;
    a.dx_part = dx.part;
    const bool summed = pieces > 1 || dx.parts > 1;
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t N = std::min(piece, a.V - v0);
        if (a.R > 0)
            if (const hipError_t e = logits<T, true>(a, v0, N, tiles_for(a.R, N, size, direct), direct, s)) return e;
        if (a.dx && a.R > 0) {
            hipError_t e = hipSuccess;
            if (dx.large) {
                if constexpr (sizeof(T) == 2) e = dx_launch<T, Large, true>(a, v0, N, summed ? v0 != 0 : -1, s);
            } else if (dx.small) {
                e = direct ? dx_launch<T, Narrow, true>(a, v0, N, summed ? v0 != 0 : -1, s)
                           : dx_launch<T, Narrow, false>(a, v0, N, summed ? v0 != 0 : -1, s);
            } else {
                e = direct ? dx_launch<T, Medium, true>(a, v0, N, summed ? v0 != 0 : -1, s)
                           : dx_launch<T, Medium, false>(a, v0, N, summed ? v0 != 0 : -1, s);
            }
            if (e) return e;
        }
        if (a.dw) {
            const int64_t chunk = dw_chunk(a.R, N, a.I);
            hipError_t e = hipSuccess;
            if (size == 2 && tiles_for(N, a.I, size, direct) == Tiles::kLarge) {
                if constexpr (sizeof(T) == 2) e = dw_launch<T, Large, true>(a, v0, N, chunk, s);
            } else if (N <= 64) {
                e = direct ? dw_launch<T, Flat, true>(a, v0, N, chunk, s)
                           : dw_launch<T, Flat, false>(a, v0, N, chunk, s);
            } else {
                e = direct ? dw_launch<T, Medium, true>(a, v0, N, chunk, s)
                           : dw_launch<T, Medium, false>(a, v0, N, chunk, s);
            }
            if (e) return e;
            if (chunk) {
                const int64_t n = N * a.I;
                loss_fold_kernel<T><<<(unsigned)std::min(tiles_of(n, kFoldElements), kMaxBlocks), kPackThreads, 0, s>>>(
                    a, v0, n, chunk);
            }
        }
    }
    if (a.dx && a.R > 0) loss_rest_kernel<T><<<pack_blocks, kPackThreads, 0, s>>>(a, summed);
    return hipGetLastError();
}

}  // namespace

// floats: the rows' maxima and inverse sums; then the list, and its length.
int64_t loss_state_bytes(int64_t R) { return whole(3 * R * 4, 8) + 8; }

// Each tile's maximum and sum, the class's logits, the blocks' counts and losses.
static int64_t forward_floats(int64_t R, int64_t V) {
    return R * tiles_of(V, V <= 64 ? 64 : 128) * 2 + R + std::max<int64_t>(1, tiles_of(R, kListRows)) +
           tiles_of(R, 8);
}

int64_t loss_workspace_bytes(int64_t R, int64_t I, int64_t V, int type) {
    return 256 + padded_bytes(R, I, V, type == SPMM_F32 ? 4 : 2) + forward_floats(R, V) * (int64_t)sizeof(float);
}

static void state_arrays(LossArgs &a, void *state) {
    a.stats = static_cast<float *>(state);
    a.rows = reinterpret_cast<int *>(a.stats + 2 * a.R);
    a.count = reinterpret_cast<int64_t *>(static_cast<char *>(state) + whole(3 * a.R * 4, 8));
}

constexpr int64_t kUnitBytes = (kUnitBlocks + 64) * 4;       // the unit, and the blocks' largest gradients

struct BackwardSizes {
    int64_t d, packed, dx_sum, dw_partial, padded;       // bytes, each whole 256s
};

static BackwardSizes backward_sizes(int64_t R, int64_t I, int64_t V, int size) {
    const int64_t piece = piece_of(R, V, size);
    BackwardSizes b;
    b.d = whole(R * piece * size, 256);
    b.packed = whole(R * padded_width(R, I, V, size) * size, 256);
    b.padded = padded_bytes(R, I, V, size);
    // the addresses are not known here: what either way of staging needs
    const int64_t parts = std::max(dx_shape(R, I, std::min(piece, V), size, true).parts,
                                   dx_shape(R, I, std::min(piece, V), size, false).parts);
    b.dx_sum = piece < V || parts > 1 ? whole(parts * R * I * 4, 256) : 0;
    b.dw_partial = 0;
    for (const int64_t n : {std::min(piece, V), V % piece}) {
        const int64_t chunk = n ? dw_chunk(R, n, I) : 0;
        if (chunk) b.dw_partial = std::max(b.dw_partial, whole(tiles_of(R, (int)chunk) * n * I * 4, 256));
    }
    return b;
}

int64_t loss_backward_workspace_bytes(int64_t R, int64_t I, int64_t V, int type) {
    const BackwardSizes b = backward_sizes(R, I, V, type == SPMM_F32 ? 4 : 2);
    return 256 + kUnitBytes + b.d + b.packed + b.dx_sum + b.dw_partial + b.padded;      // room to start on 256 bytes
}

hipError_t launch_loss(const LossArgs &args, void *state, void *workspace, int type, hipStream_t s) {
    LossArgs a = args;
    state_arrays(a, state);
    char *at = reinterpret_cast<char *>(whole((int64_t)(uintptr_t)workspace, 256));
    a.padded = at;
    a.tile_top = reinterpret_cast<float *>(at + padded_bytes(a.R, a.I, a.V, type == SPMM_F32 ? 4 : 2));
    const int64_t tiles = a.R * tiles_of(a.V, a.V <= 64 ? 64 : 128);
    a.tile_sum = a.tile_top + tiles;
    a.picked = a.tile_sum + tiles;
    a.block_count = reinterpret_cast<int *>(a.picked + a.R);
    if (!a.per_row) a.block_loss = a.picked + a.R + std::max<int64_t>(1, tiles_of(a.R, kListRows));
    if (type == SPMM_F32) return forward<float>(a, s);
    if (type == SPMM_BF16) return forward<__bf16>(a, s);
    return forward<_Float16>(a, s);
}

hipError_t launch_loss_backward(const LossArgs &args, const void *state, void *workspace, int type, hipStream_t s) {
    LossArgs a = args;
    state_arrays(a, const_cast<void *>(state));
    const BackwardSizes b = backward_sizes(a.R, a.I, a.V, type == SPMM_F32 ? 4 : 2);
    char *at = reinterpret_cast<char *>(whole((int64_t)(uintptr_t)workspace, 256));
    a.unit = reinterpret_cast<float *>(at);
    a.d = at += kUnitBytes;
    a.packed = at += b.d;
    a.dx_sum = reinterpret_cast<float *>(at += b.packed);
    a.dw_partial = reinterpret_cast<float *>(at += b.dx_sum);
    a.padded = at + b.dw_partial;
    if (type == SPMM_F32) return backward<float>(a, s);
    if (type == SPMM_BF16) return backward<__bf16>(a, s);
    return backward<_Float16>(a, s);
}

}  // namespace gspmm
