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
constexpr int kStepBytes = 128;              // of the summed index, per row of a tile

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kStep = kStepBytes / (int)sizeof(T);

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ inline int64_t uniform(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

// A tile shape: BM x BN outputs by WR x WC waves.
template <int BM_, int BN_, int WR_, int WC_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_;
    static constexpr int kWaves = WR * WC, kThreads = kWaves * kWave;
    static constexpr int kStageBytes = (BM + BN) * kStepBytes;
    static constexpr int MI = BM / WR / 32, NI = BN / WC / 32;
};
using Large = Shape<256, 256, 2, 4>;
using Medium = Shape<128, 128, 2, 2>;

// ---- LDS layout of one operand's step, B rows of the tile ----
//
// KC (summed index contiguous): B rows of 128 bytes; chunk c of row r at
// c ^ (r & 7), so that the 32 lanes that read one chunk column spread over
// the banks.
// KS (summed index = row), 16-bit: 64 rows of 2 B bytes; the 32-byte piece c
// of row k at c ^ 2 (k & 3), so that the four rows a 16-lane transposing read
// touches lie in different banks.  fp32: 32 rows of 4 B bytes, as they are.

template <typename T, bool KC, int B>
__device__ inline int chunk_offset(int outer, int chunk) {
    if constexpr (KC) return outer * kStepBytes + ((chunk ^ (outer & 7)) << 4);
    else if constexpr (sizeof(T) == 4) return outer * B * 4 + (chunk << 4);
    else return outer * B * 2 + (((chunk >> 1) ^ ((outer & 3) << 1)) << 5) + ((chunk & 1) << 4);
}

// One operand of a tile.  KC: `outer` rows (tile rows) of `inner` summed
// elements from `ptr`.  KS: `outer` summed rows of `inner` elements from ptr.
template <typename T>
struct Operand {
    const T *ptr;
    int64_t ld;
    int64_t outer;      // rows that exist
    int64_t inner;      // elements of a row that exist
    const T *end;       // end of the array
};

// Copies an operand's steps straight into LDS, 16 bytes per lane: for rows
// that start on 16 bytes and are multiples of them.  A lane's place in the
// step is fixed by its number, so the swizzle is applied to what it reads.
// What lies behind the summed range reads as zero (the lane points behind the
// buffer); tile rows (KC) and columns (KS) that do not exist read what
// follows in the same array, or zero behind its end: they only reach outputs
// that are not stored.
template <typename T, bool KC, int B, int WAVES>
struct Copy {
    static constexpr int kCopies = B * kStepBytes / 1024 / WAVES;
    static constexpr int kRowsPerCopy = KC ? 8 * WAVES : 1024 * WAVES / (B * (int)sizeof(T));

    const char *base;
    int64_t bytes;          // from base to the end of the array
    int64_t step_bytes;
    uint32_t at, next_copy; // byte offset of the lane's chunk of copy 0, and from one copy to the next
    int first;              // the lane's first summed element of copy 0 within a step
    int left;               // summed elements from the next step on

    __device__ inline Copy(const Operand<T> &o, int wave) {
        const int byte = wave * 1024 + (threadIdx.x & (kWave - 1)) * 16;
        const uint32_t row_bytes = (uint32_t)(o.ld * (int)sizeof(T));
        base = (const char *)uniform((int64_t)o.ptr);
        bytes = uniform((int64_t)((const char *)o.end - (const char *)o.ptr));
        next_copy = kRowsPerCopy * row_bytes;
        if constexpr (KC) {
            const int row = byte / kStepBytes, chunk = (byte / 16 % 8) ^ (row & 7);
            first = chunk * kPack<T>;
            left = uniform((int)o.inner);
            step_bytes = kStepBytes;
            at = row * row_bytes + chunk * 16;
        } else {
            constexpr int kRow = B * (int)sizeof(T);
            const int k = byte / kRow;
            int chunk = byte % kRow / 16;
            if constexpr (sizeof(T) == 2) chunk = (((chunk >> 1) ^ ((k & 3) << 1)) << 1) | (chunk & 1);
            first = k;
            left = uniform((int)o.outer);
            step_bytes = (int64_t)kStep<T> * uniform((int)row_bytes);
            at = k * row_bytes + chunk * 16;
        }
    }

    __device__ inline void step(char *lds, int wave) {
        const int records = (int)max(int64_t(0), min(bytes, int64_t(0x7fffffff)));
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, records, 0x00020000);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const bool in = first + (KC ? 0 : i * kRowsPerCopy) < left;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(lds + (i * WAVES + wave) * 1024), 16,
                in ? at + i * next_copy : 0x80000000u, 0, 0, 0);
        }
        base += step_bytes;
        bytes -= step_bytes;
        left -= kStep<T>;
    }
};

// The same through registers, at any width and alignment.
template <typename T, bool KC, int B, int WAVES>
__device__ inline void fetch(const Operand<T> &o, int64_t k0, Pack<T> (&r)[B * 8 / (WAVES * kWave)]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : B * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < B * 8 / (WAVES * kWave); ++i) {
        const int idx = threadIdx.x + i * WAVES * kWave, row = idx / kPerRow, c = idx % kPerRow * kPack<T>;
        const int64_t out = KC ? row : k0 + row, in = KC ? k0 + c : c;
        const int64_t n = out < o.outer ? o.inner - in : 0;
        r[i] = load_pack(o.ptr + out * o.ld + in, n);
    }
}

template <typename T, bool KC, int B, int WAVES>
__device__ inline void put(char *lds, const Pack<T> (&r)[B * 8 / (WAVES * kWave)]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : B * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < B * 8 / (WAVES * kWave); ++i) {
        const int idx = threadIdx.x + i * WAVES * kWave;
        *reinterpret_cast<Pack<T> *>(lds + chunk_offset<T, KC, B>(idx / kPerRow, idx % kPerRow)) = r[i];
    }
}

// The lane's operand values of matrix step ks for the 32 tile rows from m0:
// row m0 + lane % 32; 16-bit: summed elements ks * 16 + lane / 32 * 8 + 0..7,
// fp32: ks * 8 + lane / 32 * 4 + 0..3.
template <typename T, bool KC, int B>
__device__ inline Pack<T> frag(const char *lds, int m0, int ks) {
    const int lane = threadIdx.x & (kWave - 1), half = lane >> 5, m = m0 + (lane & 31);
    if constexpr (KC) {
        return *reinterpret_cast<const Pack<T> *>(lds + chunk_offset<T, true, B>(m, 2 * ks + half));
    } else if constexpr (sizeof(T) == 4) {
        Pack<T> r;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.v[j] = *reinterpret_cast<const float *>(lds + (ks * 8 + half * 4 + j) * B * 4 + m * 4);
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
            const int at = k * B * 2 + ((piece ^ ((k & 3) << 1)) << 5) + ((l & 3) << 3);
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

// out[0..rows) x [0..cols) of a tile = A . B over K summed elements.
template <typename T, typename OUT, typename S, bool AKC, bool BKC, bool DIRECT>
__device__ inline void tile_product(char *lds, const Operand<T> &a, const Operand<T> &b, int64_t K, OUT *out,
                                    int64_t ldo, int64_t rows, int64_t cols) {
    constexpr int MI = S::MI, NI = S::NI, kA = S::BM * kStepBytes;
    const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
    const int m0 = wave / S::WC * (MI * 32), n0 = wave % S::WC * (NI * 32);
    f32x16 acc[MI][NI] = {};
    const int steps = (int)((K + kStep<T> - 1) / kStep<T>);
    Pack<T> fa[4][MI], fb[4][NI];
    auto multiply_part = [&](int ks) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) multiply<T>(fa[ks][i], fb[ks][j], acc[i][j]);
    };
    auto read_part = [&](const char *cur, int ks) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[ks][i] = frag<T, AKC, S::BM>(cur, m0 + i * 32, ks);
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[ks][j] = frag<T, BKC, S::BN>(cur + kA, n0 + j * 32, ks);
    };
    if constexpr (DIRECT) {
        Copy<T, AKC, S::BM, S::kWaves> ca(a, wave);
        Copy<T, BKC, S::BN, S::kWaves> cb(b, wave);
        if (steps > 0) {
            ca.step(lds, wave);
            cb.step(lds + kA, wave);
        }
        __syncthreads();
        for (int t = 0; t < steps; ++t) {
            const char *cur = lds + (t & 1) * S::kStageBytes;
            char *next = lds + ((t + 1) & 1) * S::kStageBytes;
            // every read of this step goes out before the next step's copies
            // (an LDS read behind a copy would wait for it); the last of them
            // take the registers of the first part's operands
            read_part(cur, 0);
            read_part(cur, 1);
            read_part(cur, 2);
            __builtin_amdgcn_sched_barrier(0);
            multiply_part(0);
            read_part(cur, 3);
            __builtin_amdgcn_sched_barrier(0);
            if (t + 1 < steps) {
                ca.step(next, wave);
                cb.step(next + kA, wave);
            }
            __builtin_amdgcn_sched_barrier(0);
            multiply_part(1);
            multiply_part(2);
            multiply_part(3);
            __builtin_amdgcn_sched_barrier(0);       // the barrier's wait for the copies stays behind them
            __syncthreads();
        }
    } else {
        constexpr int kRegA = S::BM * 8 / S::kThreads, kRegB = S::BN * 8 / S::kThreads;
        Pack<T> ra[kRegA], rb[kRegB];
        if (steps > 0) {
            fetch<T, AKC, S::BM, S::kWaves>(a, 0, ra);
            fetch<T, BKC, S::BN, S::kWaves>(b, 0, rb);
            put<T, AKC, S::BM, S::kWaves>(lds, ra);
            put<T, BKC, S::BN, S::kWaves>(lds + kA, rb);
        }
        __syncthreads();
        for (int t = 0; t < steps; ++t) {
            const char *cur = lds + (t & 1) * S::kStageBytes;
            char *next = lds + ((t + 1) & 1) * S::kStageBytes;
            if (t + 1 < steps) {
                fetch<T, AKC, S::BM, S::kWaves>(a, (int64_t)(t + 1) * kStep<T>, ra);
                fetch<T, BKC, S::BN, S::kWaves>(b, (int64_t)(t + 1) * kStep<T>, rb);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                read_part(cur, ks);
                multiply_part(ks);
            }
            if (t + 1 < steps) {
                put<T, AKC, S::BM, S::kWaves>(next, ra);
                put<T, BKC, S::BN, S::kWaves>(next + kA, rb);
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t r = m0 + i * 32 + (lane & 31);
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j)
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

template <typename T, typename S>
__device__ inline void tile_zero(T *out, int64_t ldo, int64_t rows, int64_t cols) {
    for (int i = threadIdx.x; i < S::BM * S::BN; i += S::kThreads)
        if (i / S::BN < rows && i % S::BN < cols) out[(int64_t)(i / S::BN) * ldo + i % S::BN] = (T)0.0f;
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
template <int BM>
__device__ inline void find_tile(const SegmentArgs &a, int64_t tile, int64_t *run, int64_t *row, int64_t *end) {
    const int lane = threadIdx.x & (kWave - 1);
    *run = -1;
    for (int64_t v0 = 0; v0 < a.E + 2; v0 += kWave) {
        const int64_t v = v0 + lane;
        const int64_t lo = v < a.E + 2 ? run_bound(a, v) : 0, hi = v < a.E + 2 ? run_bound(a, v + 1) : 0;
        const int64_t mine = hi > lo ? (hi - lo + BM - 1) / BM : 0;
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
            *row = __shfl(lo, at, kWave) + (tile - before) * BM;
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

template <typename T, typename S, bool TRANSPOSED, bool DIRECT>
__global__ __launch_bounds__(S::kThreads) void segment_kernel(SegmentArgs a, int64_t col_tiles, int64_t total) {
    __shared__ __attribute__((aligned(1024))) char lds[2 * S::kStageBytes];
    const int64_t K = TRANSPOSED ? a.O : a.I, N = TRANSPOSED ? a.I : a.O;
    const T *in = (const T *)(TRANSPOSED ? a.dy : a.x), *w = (const T *)a.w;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int64_t t = xcd_order(id, total), n0 = t % col_tiles * S::BN;
        int64_t run, row, end;
        find_tile<S::BM>(a, t / col_tiles, &run, &row, &end);
        run = uniform(run);
        if (run < 0) continue;
        row = uniform(row);
        end = uniform(end);
        T *out = (T *)a.y + row * N + n0;
        const int64_t rows = end - row;
        if (run == 0 || run > a.E) {
            tile_zero<T, S>(out, N, rows, N - n0);
            continue;
        }
        Operand<T> A, B;
        A.ptr = in + row * K;
        A.ld = K;
        A.outer = rows;
        A.inner = K;
        A.end = in + a.R * K;
        const T *we = w + (run - 1) * a.I * a.O;
        B.end = w + a.E * a.I * a.O;
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
        tile_product<T, T, S, true, TRANSPOSED, DIRECT>(lds, A, B, K, out, N, rows, N - n0);
    }
}

// dw: tile (segment, split of its rows, tile of [I, O]); splits > 1 write fp32
// partial sums [splits][E][I][O].
template <typename T, typename OUT, typename S, bool DIRECT>
__global__ __launch_bounds__(S::kThreads) void segment_dw_kernel(SegmentArgs a, OUT *dst, int64_t row_tiles,
                                                                 int64_t col_tiles, int64_t splits, int64_t total) {
    __shared__ __attribute__((aligned(1024))) char lds[2 * S::kStageBytes];
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        int64_t t = xcd_order(id, total);
        const int64_t n0 = t % col_tiles * S::BN;
        t /= col_tiles;
        const int64_t m0 = t % row_tiles * S::BM;
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
        A.end = (const T *)a.x + a.R * a.I;
        B.ptr = (const T *)a.dy + (lo + k0) * a.O + n0;
        B.ld = a.O;
        B.outer = k1 - k0;
        B.inner = a.O - n0;
        B.end = (const T *)a.dy + a.R * a.O;
        __syncthreads();
        tile_product<T, OUT, S, false, false, DIRECT>(lds, A, B, k1 - k0, dst + ((s * a.E + e) * a.I + m0) * a.O + n0,
                                                      a.O, a.I - m0, a.O - n0);
    }
}

constexpr int kFoldThreads = 256;

template <typename T>
__global__ __launch_bounds__(kFoldThreads) void segment_fold_kernel(const float *partial, T *out, int64_t n,
                                                                    int64_t splits) {
    for (int64_t i = (int64_t)blockIdx.x * kFoldThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kFoldThreads) {
        float t = 0.0f;
        for (int64_t s = 0; s < splits; ++s) t += partial[s * n + i];
        out[i] = (T)t;
    }
}

int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

constexpr int64_t kMaxBlocks = 1 << 20;
constexpr int64_t kUnits = 256;                      // compute units

// The copy into LDS needs rows of whole 16-byte groups, from a 16-byte
// address, and 32-bit offsets within a tile's rows.
bool direct_rows(const void *p, int64_t width, int size) {
    return (uintptr_t)p % 16 == 0 && width * size % 16 == 0 && width * size * 320 < (int64_t(1) << 31);
}

// 256 x 256 tiles when there are enough of them to fill the chip.
bool large_tiles(int64_t tiles, int size, bool direct) { return direct && size == 2 && tiles >= 2 * kUnits; }

// Splits of each segment's rows in dw: enough tiles to fill the chip, but at
// least 8 steps of rows on average in each.
struct DwShape {
    bool large;
    int64_t row_tiles, col_tiles, splits;
};

DwShape dw_shape(int64_t R, int64_t E, int64_t I, int64_t O, int size, bool direct) {
    DwShape d;
    d.large = large_tiles(E * tiles_of(I, 256) * tiles_of(O, 256), size, direct);
    const int tile = d.large ? 256 : 128;
    d.row_tiles = tiles_of(I, tile);
    d.col_tiles = tiles_of(O, tile);
    const int64_t tiles = E * d.row_tiles * d.col_tiles;
    const int64_t want = (4 * kUnits + tiles - 1) / tiles, most = std::max<int64_t>(1, R / E / (8 * kStepBytes / size));
    d.splits = d.large ? 1 : std::max<int64_t>(1, std::min(want, most));
    return d;
}

template <typename T, typename S, bool DIRECT>
hipError_t segment_launch(const SegmentArgs &a, bool transposed, hipStream_t s) {
    // each run adds at most one partial tile
    const int64_t row_tiles = a.R / S::BM + a.E + 2, col_tiles = tiles_of(transposed ? a.I : a.O, S::BN);
    const int64_t total = row_tiles * col_tiles;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    if (transposed) segment_kernel<T, S, true, DIRECT><<<blocks, S::kThreads, 0, s>>>(a, col_tiles, total);
    else segment_kernel<T, S, false, DIRECT><<<blocks, S::kThreads, 0, s>>>(a, col_tiles, total);
    return hipGetLastError();
}

template <typename T>
hipError_t segment(const SegmentArgs &a, bool transposed, hipStream_t s) {
    if (a.R == 0) return hipSuccess;
    const bool direct = direct_rows(transposed ? a.dy : a.x, transposed ? a.O : a.I, sizeof(T)) &&
                        direct_rows(a.w, a.O, sizeof(T)) && a.I * (int)sizeof(T) % 16 == 0;
    const int64_t tiles = tiles_of(a.R, 256) * tiles_of(transposed ? a.I : a.O, 256);
    if constexpr (sizeof(T) == 2)
        if (large_tiles(tiles, sizeof(T), direct)) return segment_launch<T, Large, true>(a, transposed, s);
    return direct ? segment_launch<T, Medium, true>(a, transposed, s)
                  : segment_launch<T, Medium, false>(a, transposed, s);
}

template <typename T, typename OUT>
hipError_t segment_dw_launch(const SegmentArgs &a, OUT *dst, const DwShape &d, bool direct, hipStream_t s) {
    const int64_t total = a.E * d.splits * d.row_tiles * d.col_tiles;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    if constexpr (sizeof(T) == 2) {
        if (d.large) {
            segment_dw_kernel<T, OUT, Large, true><<<blocks, Large::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                     d.splits, total);
            return hipGetLastError();
        }
    }
    if (direct)
        segment_dw_kernel<T, OUT, Medium, true><<<blocks, Medium::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                   d.splits, total);
    else
        segment_dw_kernel<T, OUT, Medium, false><<<blocks, Medium::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                    d.splits, total);
    return hipGetLastError();
}

template <typename T>
hipError_t segment_dw(const SegmentArgs &a, hipStream_t s) {
    const bool direct = direct_rows(a.x, a.I, sizeof(T)) && direct_rows(a.dy, a.O, sizeof(T));
    const DwShape d = dw_shape(a.R, a.E, a.I, a.O, sizeof(T), direct);
    if (d.splits == 1) return segment_dw_launch<T, T>(a, (T *)a.y, d, direct, s);
    if (const hipError_t e = segment_dw_launch<T, float>(a, a.partial, d, direct, s)) return e;
    const int64_t n = a.E * a.I * a.O;
    segment_fold_kernel<T><<<(unsigned)std::min((n + kFoldThreads - 1) / kFoldThreads, kMaxBlocks), kFoldThreads, 0,
                             s>>>(a.partial, (T *)a.y, n, d.splits);
    return hipGetLastError();
}

}  // namespace

int64_t segment_workspace_floats(int64_t R, int64_t E, int64_t I, int64_t O, int type) {
    // the addresses are not known here: what either way of staging needs
    int64_t splits = 1;
    for (const bool direct : {false, true})
        splits = std::max(splits, dw_shape(R, E, I, O, type == SPMM_F32 ? 4 : 2, direct).splits);
    return splits == 1 ? 0 : splits * E * I * O;
}

hipError_t launch_segment(const SegmentArgs &a, bool transposed, int type, hipStream_t s) {
    if (type == SPMM_F32) return segment<float>(a, transposed, s);
    if (type == SPMM_BF16) return segment<__bf16>(a, transposed, s);
    return segment<_Float16>(a, transposed, s);
}

hipError_t launch_segment_dw(const SegmentArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return segment_dw<float>(a, s);
    if (type == SPMM_BF16) return segment_dw<__bf16>(a, s);
    return segment_dw<_Float16>(a, s);
}

}  // namespace gspmm
