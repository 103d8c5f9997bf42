// Segment product: rows sorted by expert (or node type) times that expert's
// matrix, and its two gradients.  For offsets[e] <= r < offsets[e + 1]:
//
//   y[r]  = x[r] . w[e]            x [R, I], w [E, I, O], y [R, O]
//   dx[r] = dy[r] . w[e]^T
//   dw[e] = x_e^T . dy_e           sum over the rows of e
//
// and zero rows of y and dx outside [offsets[0], offsets[E]).  One tile kernel
// on the matrix cores serves all three; they differ in which operands hold
// the summed index contiguously (x, dy in the first two, w in dx) and which
// hold it as the row (w in y, both in dw).  Products accumulate in fp32.
//
// A block of 4 waves computes a 128 x 128 tile, each wave 64 x 64, with steps
// of 128 bytes of the summed index (64 16-bit or 32 fp32 elements).  Both
// operands' steps are staged in LDS, double buffered, in the orientation they
// have in memory; operands whose rows are the summed index are turned by the
// transposing LDS read (16-bit) or read element by element (fp32).
//
// The row operands' tiles come from the segment bounds on the device: tile
// number -> segment by a wave-wide scan over the segments' tile counts, so no
// size crosses to the host and a captured call follows new offsets.
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kStepBytes = 128;
constexpr int kChunks = kTile * kStepBytes / 16;     // 16-byte chunks of one operand's step

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kStep = kStepBytes / (int)sizeof(T);

// ---- LDS layout of one operand's step ----
//
// KC (summed index contiguous): 128 rows of 128 bytes; chunk c of row r at
// c ^ (r & 7), so that the 32 lanes that read one chunk column spread over
// the banks.
// KS (summed index = row), 16-bit: 64 rows of 256 bytes; the 32-byte piece c
// of row k at c ^ 2 (k & 3), so that the four rows a 16-lane transposing read
// touches lie in different banks.  fp32: 32 rows of 512 bytes, as they are.

template <typename T, bool KC>
__device__ inline int chunk_offset(int outer, int chunk) {
    if constexpr (KC) return outer * kStepBytes + ((chunk ^ (outer & 7)) << 4);
    else if constexpr (sizeof(T) == 4) return outer * kTile * 4 + (chunk << 4);
    else return outer * kTile * 2 + (((chunk >> 1) ^ ((outer & 3) << 1)) << 5) + ((chunk & 1) << 4);
}

// One operand of a tile.  KC: `outer` rows (tile rows) of `inner` summed
// elements from `ptr`.  KS: `outer` summed rows of `inner` elements from ptr.
template <typename T>
struct Operand {
    const T *ptr;
    int64_t ld;
    int64_t outer;      // rows that exist
    int64_t inner;      // elements of a row that exist
};

template <typename T, bool KC>
__device__ inline void fetch(const Operand<T> &o, int64_t k0, Pack<T> (&r)[kChunks / kThreads]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : kTile * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < kChunks / kThreads; ++i) {
        const int idx = threadIdx.x + i * kThreads, row = idx / kPerRow, c = idx % kPerRow * kPack<T>;
        const int64_t out = KC ? row : k0 + row, in = KC ? k0 + c : c;
        const int64_t n = out < o.outer ? o.inner - in : 0;
        r[i] = load_pack(o.ptr + out * o.ld + in, n);
    }
}

template <typename T, bool KC>
__device__ inline void put(char *lds, const Pack<T> (&r)[kChunks / kThreads]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : kTile * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < kChunks / kThreads; ++i) {
        const int idx = threadIdx.x + i * kThreads;
        *reinterpret_cast<Pack<T> *>(lds + chunk_offset<T, KC>(idx / kPerRow, idx % kPerRow)) = r[i];
    }
}

// The lane's operand values of matrix step ks for the 32 tile rows from m0:
// row m0 + lane % 32; 16-bit: summed elements ks * 16 + lane / 32 * 8 + 0..7,
// fp32: ks * 8 + lane / 32 * 4 + 0..3.
template <typename T, bool KC>
__device__ inline Pack<T> frag(const char *lds, int m0, int ks) {
    const int lane = threadIdx.x & (kWave - 1), half = lane >> 5, m = m0 + (lane & 31);
    if constexpr (KC) {
        return *reinterpret_cast<const Pack<T> *>(lds + chunk_offset<T, true>(m, 2 * ks + half));
    } else if constexpr (sizeof(T) == 4) {
        Pack<T> r;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.v[j] = *reinterpret_cast<const float *>(lds + (ks * 8 + half * 4 + j) * kTile * 4 + m * 4);
        return r;
    } else {
        // lane l of a 16-lane group points at 4 elements of summed row l / 4
        // and receives element l of the rows 0..3
        const int l = lane & 15, piece = (m0 >> 4) + ((lane >> 4) & 1);
        struct {
            i16x4 lo, hi;
        } both;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = ks * 16 + half * 8 + q * 4 + (l >> 2);
            const int at = k * kTile * 2 + ((piece ^ ((k & 3) << 1)) << 5) + ((l & 3) << 3);
            auto *p = (__attribute__((address_space(3))) i16x4 *)(lds + at);
            (q ? both.hi : both.lo) = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
        }
        return __builtin_bit_cast(Pack<T>, both);
    }
}

// acc += a . b with a's 32 rows in the lanes and b's 32 rows in the registers
// (operands exchanged): lane l holds row l % 32 of a against rows
// 8 (i / 4) + 4 (l / 32) + i % 4 of b, i = 0..15.
template <typename T>
__device__ inline void multiply(const Pack<T> &a, const Pack<T> &b, f32x16 &acc) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(b.v[j], a.v[j], acc, 0, 0, 0);
    } else if constexpr (__is_same(T, __bf16)) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a),
                                                      acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), acc,
                                                     0, 0, 0);
    }
}

// out[0..rows) x [0..cols) of a 128 x 128 tile = A . B over K summed elements.
template <typename T, typename OUT, bool AKC, bool BKC>
__device__ inline void tile_product(char *lds, const Operand<T> &a, const Operand<T> &b, int64_t K, OUT *out,
                                    int64_t ldo, int64_t rows, int64_t cols) {
    constexpr int kBytes = kChunks * 16;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int m0 = (wave >> 1) * 64, n0 = (wave & 1) * 64;
    f32x16 acc[2][2] = {};
    const int64_t steps = (K + kStep<T> - 1) / kStep<T>;
    Pack<T> ra[kChunks / kThreads], rb[kChunks / kThreads];
    if (steps > 0) {
        fetch<T, AKC>(a, 0, ra);
        fetch<T, BKC>(b, 0, rb);
        put<T, AKC>(lds, ra);
        put<T, BKC>(lds + kBytes, rb);
    }
    __syncthreads();
    for (int64_t t = 0; t < steps; ++t) {
        const char *cur = lds + (t & 1) * 2 * kBytes;
        char *next = lds + ((t + 1) & 1) * 2 * kBytes;
        if (t + 1 < steps) {
            fetch<T, AKC>(a, (t + 1) * kStep<T>, ra);
            fetch<T, BKC>(b, (t + 1) * kStep<T>, rb);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            Pack<T> fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = frag<T, AKC>(cur, m0 + i * 32, ks);
                fb[i] = frag<T, BKC>(cur + kBytes, n0 + i * 32, ks);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) multiply<T>(fa[i], fb[j], acc[i][j]);
        }
        if (t + 1 < steps) {
            put<T, AKC>(next, ra);
            put<T, BKC>(next + kBytes, rb);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = m0 + i * 32 + (lane & 31);
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t c = n0 + j * 32 + q * 8 + (lane >> 5) * 4;
                struct {
                    OUT v[4];
                } o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o.v[e] = (OUT)acc[i][j][q * 4 + e];
                OUT *p = out + r * ldo + c;
                if (c + 4 <= cols) __builtin_memcpy(p, &o, sizeof(o));
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < cols) p[e] = o.v[e];
            }
    }
}

template <typename T>
__device__ inline void tile_zero(T *out, int64_t ldo, int64_t rows, int64_t cols) {
    if (cols > kTile) cols = kTile;
    if (rows > kTile) rows = kTile;
    for (int i = threadIdx.x; i < kTile * kTile; i += kThreads)
        if (i / kTile < rows && i % kTile < cols) out[(i / kTile) * ldo + i % kTile] = (T)0.0f;
}

// Bound i of the E + 2 runs of rows: those before the first segment, the
// segments, those behind the last one.
__device__ inline int64_t run_bound(const SegmentArgs &a, int64_t i) {
    if (i <= 0) return 0;
    if (i > a.E + 1) return a.R;
    const int64_t b = a.offsets[i - 1];
    return b < 0 ? 0 : b > a.R ? a.R : b;
}

// Run and first row of row tile `tile`; run < 0: there is no such tile.
// Every wave finds it by itself: 64 runs at a time, a scan of their tiles.
__device__ inline void find_tile(const SegmentArgs &a, int64_t tile, int64_t *run, int64_t *row, int64_t *end) {
    const int lane = threadIdx.x & (kWave - 1);
    *run = -1;
    for (int64_t v0 = 0; v0 < a.E + 2; v0 += kWave) {
        const int64_t v = v0 + lane;
        const int64_t lo = v < a.E + 2 ? run_bound(a, v) : 0, hi = v < a.E + 2 ? run_bound(a, v + 1) : 0;
        const int64_t mine = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const int64_t up = __shfl_up(incl, o, kWave);
            if (lane >= o) incl += up;
        }
        const uint64_t past = __ballot(incl > tile);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            const int64_t before = __shfl(incl - mine, at, kWave);
            *run = v0 + at;
            *row = __shfl(lo, at, kWave) + (tile - before) * kTile;
            *end = __shfl(hi, at, kWave);
            return;
        }
        tile -= __shfl(incl, kWave - 1, kWave);
    }
}

// Blocks are dealt to the 8 XCDs in turn: give each XCD a run of consecutive
// tiles, whose operands then meet in one L2.
__device__ inline int64_t xcd_order(int64_t id, int64_t total) {
    const int64_t per = total / 8, extra = total % 8, x = id % 8, at = id / 8;
    return x * per + (x < extra ? x : extra) + at;
}

template <typename T, bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void segment_kernel(SegmentArgs a, int64_t col_tiles, int64_t total) {
    __shared__ __attribute__((aligned(16))) char lds[4 * kChunks * 16];
    const int64_t K = TRANSPOSED ? a.O : a.I, N = TRANSPOSED ? a.I : a.O;
    const T *in = (const T *)(TRANSPOSED ? a.dy : a.x), *w = (const T *)a.w;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int64_t t = xcd_order(id, total), n0 = t % col_tiles * kTile;
        int64_t run, row, end;
        find_tile(a, t / col_tiles, &run, &row, &end);
        if (run < 0) continue;
        T *out = (T *)a.y + row * N + n0;
        const int64_t rows = end - row;
        if (run == 0 || run > a.E) {
            tile_zero(out, N, rows, N - n0);
            continue;
        }
        Operand<T> A, B;
        A.ptr = in + row * K;
        A.ld = K;
        A.outer = rows;
        A.inner = K;
        const T *we = w + (run - 1) * a.I * a.O;
        if (TRANSPOSED) {                            // rows of w[e] are output columns
            B.ptr = we + n0 * a.O;
            B.ld = a.O;
            B.outer = N - n0;
            B.inner = K;
        } else {                                     // rows of w[e] are summed
            B.ptr = we + n0;
            B.ld = a.O;
            B.outer = K;
            B.inner = N - n0;
        }
        __syncthreads();
        tile_product<T, T, true, TRANSPOSED>(lds, A, B, K, out, N, rows, N - n0);
    }
}

// dw: tile (segment, split of its rows, tile of [I, O]); splits > 1 write fp32
// partial sums [splits][E][I][O].
template <typename T, typename OUT>
__global__ __launch_bounds__(kThreads) void segment_dw_kernel(SegmentArgs a, OUT *dst, int64_t row_tiles,
                                                              int64_t col_tiles, int64_t splits, int64_t total) {
    __shared__ __attribute__((aligned(16))) char lds[4 * kChunks * 16];
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        int64_t t = xcd_order(id, total);
        const int64_t n0 = t % col_tiles * kTile;
        t /= col_tiles;
        const int64_t m0 = t % row_tiles * kTile;
        t /= row_tiles;
        const int64_t s = t % splits, e = t / splits;
        const int64_t lo = run_bound(a, e + 1);
        int64_t len = run_bound(a, e + 2) - lo;
        if (len < 0) len = 0;
        const int64_t steps = (len + kStep<T> - 1) / kStep<T>, per = (steps + splits - 1) / splits * kStep<T>;
        const int64_t k0 = min(len, s * per), k1 = min(len, k0 + per);
        Operand<T> A, B;
        A.ptr = (const T *)a.x + (lo + k0) * a.I + m0;
        A.ld = a.I;
        A.outer = k1 - k0;
        A.inner = a.I - m0;
        B.ptr = (const T *)a.dy + (lo + k0) * a.O + n0;
        B.ld = a.O;
        B.outer = k1 - k0;
        B.inner = a.O - n0;
        __syncthreads();
        tile_product<T, OUT, false, false>(lds, A, B, k1 - k0, dst + ((s * a.E + e) * a.I + m0) * a.O + n0, a.O,
                                           a.I - m0, a.O - n0);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void segment_fold_kernel(const float *partial, T *out, int64_t n,
                                                                int64_t splits) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        float t = 0.0f;
        for (int64_t s = 0; s < splits; ++s) t += partial[s * n + i];
        out[i] = (T)t;
    }
}

int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

// Splits of each segment's rows in dw: enough tiles to fill the chip twice,
// but at least 8 steps of rows on average in each.
int64_t dw_splits(int64_t R, int64_t E, int64_t I, int64_t O, int type) {
    const int64_t tiles = E * tiles_of(I) * tiles_of(O), step = type == SPMM_F32 ? kStep<float> : kStep<_Float16>;
    const int64_t want = (1024 + tiles - 1) / tiles, most = std::max<int64_t>(1, R / E / (8 * step));
    return std::max<int64_t>(1, std::min(want, most));
}

constexpr int64_t kMaxBlocks = 1 << 20;

template <typename T>
hipError_t segment(const SegmentArgs &a, bool transposed, hipStream_t s) {
    // each run adds at most one partial tile
    const int64_t row_tiles = a.R / kTile + a.E + 2, col_tiles = tiles_of(transposed ? a.I : a.O);
    if (a.R == 0) return hipSuccess;
    const int64_t total = row_tiles * col_tiles;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    if (transposed) segment_kernel<T, true><<<blocks, kThreads, 0, s>>>(a, col_tiles, total);
    else segment_kernel<T, false><<<blocks, kThreads, 0, s>>>(a, col_tiles, total);
    return hipGetLastError();
}

template <typename T>
hipError_t segment_dw(const SegmentArgs &a, int type, hipStream_t s) {
    const int64_t splits = dw_splits(a.R, a.E, a.I, a.O, type);
    const int64_t rt = tiles_of(a.I), ct = tiles_of(a.O), total = a.E * splits * rt * ct;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    if (splits == 1) {
        segment_dw_kernel<T, T><<<blocks, kThreads, 0, s>>>(a, (T *)a.y, rt, ct, splits, total);
        return hipGetLastError();
    }
    segment_dw_kernel<T, float><<<blocks, kThreads, 0, s>>>(a, a.partial, rt, ct, splits, total);
    if (const hipError_t e = hipGetLastError()) return e;
    const int64_t n = a.E * a.I * a.O;
    segment_fold_kernel<T><<<(unsigned)std::min((n + kThreads - 1) / kThreads, kMaxBlocks), kThreads, 0, s>>>(
        a.partial, (T *)a.y, n, splits);
    return hipGetLastError();
}

}  // namespace

int64_t segment_workspace_floats(int64_t R, int64_t E, int64_t I, int64_t O, int type) {
    const int64_t splits = dw_splits(R, E, I, O, type);
    return splits == 1 ? 0 : splits * E * I * O;
}

hipError_t launch_segment(const SegmentArgs &a, bool transposed, int type, hipStream_t s) {
    if (type == SPMM_F32) return segment<float>(a, transposed, s);
    if (type == SPMM_BF16) return segment<__bf16>(a, transposed, s);
    return segment<_Float16>(a, transposed, s);
}

hipError_t launch_segment_dw(const SegmentArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return segment_dw<float>(a, type, s);
    if (type == SPMM_BF16) return segment_dw<__bf16>(a, type, s);
    return segment_dw<_Float16>(a, type, s);
}

}  // namespace gspmm
