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
// A block computes one tile of the output, in steps of 64 bytes of the summed
// index (32 16-bit or 16 fp32 elements).  Both operands' steps are copied
// straight into LDS in the orientation they have in memory, four steps ahead
// of the matrix instructions; operands whose rows are the summed index are
// turned by the transposing LDS read (16-bit) or read element by element
// (fp32).
//
// The row operands' tiles come from the segment bounds on the device: tile
// number -> segment by a wave-wide scan over the segments' tile counts, or by a
// search where there are many, so no size crosses to the host and a captured
// call follows new offsets.
//
// Measured, medians of the kernels alone under the profiler: 65,536 rows in 32
// segments, 1024 x 2048 bf16, y 310 us, dx 312 us (0.88 PFLOP/s), dw 259 us
// (1.06), matrix cores 45%, 45% and 52% busy: a block to a unit, so the first
// copies and the last stores of a tile are not covered.  150,001 rows in 7, 128 x
// 256 fp32: y 124, dx 110, dw 98 + 11 us (79 to 101 TFLOP/s of the 154 that a
// large fp32 product reaches).  96 rows in 16, 1024 x 2048 bf16: 14 us, the
// weights' 67 MB at 4.9 TB/s.
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kWave = 64;
constexpr int kStepBytes = 64;               // of the summed index, per row of a tile
constexpr int kChunks = kStepBytes / 16;     // 16-byte chunks of them
constexpr int kParts = kStepBytes / 32;      // matrix steps of them
constexpr int kStages = 4;                   // steps held in LDS

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kStep = kStepBytes / (int)sizeof(T);

// LDS addresses keep their address space, and with it the name of the array
// they point into (see Stages).
typedef __attribute__((address_space(3))) char LdsByte;
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

template <typename V>
__device__ inline V lds_load(LdsByte *p) {
    return __builtin_bit_cast(V, *(__attribute__((address_space(3))) i32x4 *)p);
}

template <typename V>
__device__ inline void lds_store(LdsByte *p, const V &v) {
    *(__attribute__((address_space(3))) i32x4 *)p = __builtin_bit_cast(i32x4, v);
}

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
// KC (summed index contiguous): B rows of 64 bytes; chunk c of row r at
// c ^ (r / 4 & 3), so that 16 lanes that read one chunk column of 16 rows
// cover all 64 banks once.
// KS (summed index = row), 16-bit: 32 rows of 2 B bytes; the 32-byte piece c
// of row k at c ^ 2 (k & 3), so that the four rows a 16-lane transposing read
// touches lie in different banks.  fp32: 16 rows of 4 B bytes, as they are.

template <typename T, bool KC, int B>
__device__ inline int chunk_offset(int outer, int chunk) {
    if constexpr (KC) return outer * kStepBytes + ((chunk ^ (outer >> 2 & 3)) << 4);
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
    static constexpr int kRowsPerCopy = KC ? 1024 / kStepBytes * WAVES : 1024 * WAVES / (B * (int)sizeof(T));

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
            const int row = byte / kStepBytes, chunk = (byte / 16 % kChunks) ^ (row >> 2 & 3);
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

    __device__ inline void step(LdsByte *lds, int wave) {
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

// The same through registers, at any width and alignment.  Steps ahead of the
// last one load whole packs: a tile row (KC) that does not exist repeats the
// last one, and a pack of columns (KS) that crosses the end of its row reads
// on into the next, which exists; both only reach outputs that are not
// stored.  The last step, and every step of rows below a pack, loads exactly
// the elements that exist.
template <typename T, bool KC, int B, int WAVES, bool WHOLE>
__device__ inline void fetch(const Operand<T> &o, int64_t k0, Pack<T> (&r)[B * kChunks / (WAVES * kWave)]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : B * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < B * kChunks / (WAVES * kWave); ++i) {
        const int idx = threadIdx.x + i * WAVES * kWave, row = idx / kPerRow, c = idx % kPerRow * kPack<T>;
        if constexpr (WHOLE) {
            const int64_t out = KC ? min(int64_t(row), o.outer - 1) : k0 + row;
            const int64_t in = KC ? k0 + c : min(int64_t(c), o.inner - 1);
            r[i] = load_pack(o.ptr + out * o.ld + in);
        } else {
            const int64_t out = KC ? row : k0 + row, in = KC ? k0 + c : c;
            const int64_t n = out < o.outer ? o.inner - in : 0;
            r[i] = load_pack(o.ptr + out * o.ld + in, n);
        }
    }
}

template <typename T, bool KC, int B, int WAVES>
__device__ inline void put(LdsByte *lds, const Pack<T> (&r)[B * kChunks / (WAVES * kWave)]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : B * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < B * kChunks / (WAVES * kWave); ++i) {
        const int idx = threadIdx.x + i * WAVES * kWave;
        lds_store(lds + chunk_offset<T, KC, B>(idx / kPerRow, idx % kPerRow), r[i]);
    }
}

// The lane's operand values of matrix step ks for the 32 tile rows from
// m0 + 32 i: row m0 + 32 i + lane % 32; 16-bit: summed elements ks * 16 +
// lane / 32 * 8 + 0..7, fp32: ks * 8 + lane / 32 * 4 + 0..3.
//
// Offsets that depend on the lane are computed once and hidden from the
// optimiser, so that an address is a stage, a lane's offset and a constant:
// longer chains lose the stage's name (see Stages).
template <typename T, bool KC, int B, int COUNT>
struct Reader {
    static constexpr bool kTurned = !KC && sizeof(T) == 2;
    int at[KC ? kParts : kTurned ? COUNT : 1];

    __device__ inline Reader(int m0) {
        const int lane = threadIdx.x & (kWave - 1), half = lane >> 5, m = m0 + (lane & 31);
        if constexpr (KC) {
#pragma unroll
            for (int ks = 0; ks < kParts; ++ks) at[ks] = chunk_offset<T, true, B>(m, 2 * ks + half);
        } else if constexpr (kTurned) {
            // lane l of a 16-lane group points at 4 elements of summed row
            // l / 4 and receives element l of the rows 0..3
            const int l = lane & 15, k = half * 8 + (l >> 2);
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const int piece = (m0 >> 4) + 2 * i + ((lane >> 4) & 1);
                at[i] = k * B * 2 + ((piece ^ ((k & 3) << 1)) << 5) + ((l & 3) << 3);
            }
        } else {
            at[0] = half * 4 * B * 4 + m * 4;
        }
#pragma unroll
        for (int &o : at) asm volatile("" : "+v"(o));
    }

    template <int BASE>
    __device__ inline Pack<T> read(LdsByte *stage, int i, int ks) const {
        if constexpr (KC) {
            return lds_load<Pack<T>>(stage + at[ks] + (BASE + i * 32 * kStepBytes));
        } else if constexpr (kTurned) {
            struct {
                i16x4 lo, hi;
            } both;
            typedef __attribute__((address_space(3))) i16x4 LdsFour;
            LdsByte *p = stage + at[i] + (BASE + ks * 16 * B * 2);
            both.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsFour *)p);
            both.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsFour *)(p + 4 * B * 2));
            return __builtin_bit_cast(Pack<T>, both);
        } else {
            Pack<T> r;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r.v[j] = *(__attribute__((address_space(3))) float *)(stage + at[0] +
                                                                      (BASE + (ks * 8 + j) * B * 4 + i * 32 * 4));
            return r;
        }
    }
};

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

// Waits until at most N of the wave's copies are in flight and its LDS reads
// are back, then for the block; LDS accesses stay on their side of it.
template <int N>
__device__ inline void wait_copies() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The stages of a block.  Each is an array of its own, named at compile time
// by the unrolled loop below: a read of one stage then does not wait for the
// copies into the others.
struct Stages {
    LdsByte *at[kStages];
};

#define SEGMENT_STAGES(name, bytes)                                                                 \
    __shared__ __attribute__((aligned(1024))) char name##0[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##1[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##2[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##3[bytes];                                  \
    const Stages name = {{(LdsByte *)name##0, (LdsByte *)name##1, (LdsByte *)name##2, (LdsByte *)name##3}}

// out[0..rows) x [0..cols) of a tile = A . B over K summed elements.
template <typename T, typename OUT, typename S, bool AKC, bool BKC, bool DIRECT>
__device__ inline void tile_product(const Stages &lds, const Operand<T> &a, const Operand<T> &b, int64_t K, OUT *out,
                                    int64_t ldo, int64_t rows, int64_t cols, bool stream) {
    constexpr int MI = S::MI, NI = S::NI, kA = S::BM * kStepBytes;
    const int wave = uniform((int)threadIdx.x / kWave);
    const int m0 = wave / S::WC * (MI * 32), n0 = wave % S::WC * (NI * 32);
    f32x16 acc[MI][NI] = {};
    const int steps = (int)((K + kStep<T> - 1) / kStep<T>);
    struct Operands {
        Pack<T> a[kParts][MI], b[kParts][NI];
    };
    const Reader<T, AKC, S::BM, MI> read_a(m0);
    const Reader<T, BKC, S::BN, NI> read_b(n0);
    auto read_step = [&](LdsByte *from, Operands &to) {
#pragma unroll
        for (int ks = 0; ks < kParts; ++ks) {
#pragma unroll
            for (int j = 0; j < NI; ++j) to.b[ks][j] = read_b.template read<kA>(from, j, ks);
#pragma unroll
            for (int i = 0; i < MI; ++i) to.a[ks][i] = read_a.template read<0>(from, i, ks);
        }
    };
    auto multiply_step = [&](const Operands &o) {
#pragma unroll
        for (int ks = 0; ks < kParts; ++ks)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) multiply<T>(o.a[ks][i], o.b[ks][j], acc[i][j]);
    };
    if constexpr (DIRECT) {
        // In step t the matrix instructions work on registers read in step
        // t - 1, stage t + 1 is read, and the copies of step t + 4 go into
        // stage t.  Copies behind the last step read nothing and write zeros,
        // so that every step waits for the same number of them; the loop body
        // has no branch, so that a read waits for the copies of its own stage.
        Copy<T, AKC, S::BM, S::kWaves> ca(a, wave);
        Copy<T, BKC, S::BN, S::kWaves> cb(b, wave);
        constexpr int kCopies = decltype(ca)::kCopies + decltype(cb)::kCopies;
        // dw's large tiles have twice the LDS reads of y's: one copy (0x20) and
        // an even share of the reads (0x100) are put before each product (0x8)
        // (loops of one call, 65,536 rows in 32 segments, 1024 x 2048 bf16: 282 ->
        // 271 us, in 8, 2048 x 4096: 882 -> 853 us).  y and dx gain 3% or lose it by the
        // sizes, and keep the compiler's order.
        constexpr bool kSpread = S::BM == 256 && !AKC && !BKC;
        constexpr int kProducts = kParts * MI * NI, kReads = kParts * (MI + NI) * 2;
        constexpr int kPerProduct = (kReads + kProducts - 1) / kProducts;
        Operands set[2];
        auto copy_step = [&](LdsByte *to) {
            ca.step(to, wave);
            cb.step(to + kA, wave);
        };
        auto one_step = [&](int u) {
            wait_copies<(kStages - 2) * kCopies>();
            copy_step(lds.at[u]);
            read_step(lds.at[(u + 1) % kStages], set[(u + 1) & 1]);
            multiply_step(set[u & 1]);
            if constexpr (kSpread) {
#pragma unroll
                for (int i = 0; i < kProducts; ++i) {
                    if (i * kPerProduct < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kPerProduct, 0);
                    if (i < kCopies) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int u = 0; u < kStages; ++u) copy_step(lds.at[u]);
        wait_copies<(kStages - 1) * kCopies>();
        read_step(lds.at[0], set[0]);
        int t = steps;
        for (; t >= kStages; t -= kStages) {
#pragma unroll
            for (int u = 0; u < kStages; ++u) one_step(u);
        }
        if (t > 0) {
            one_step(0);
            if (t > 1) {
                one_step(1);
                if (t > 2) one_step(2);
            }
        }
        wait_copies<0>();
    } else {
        constexpr int kRegA = S::BM * kChunks / S::kThreads, kRegB = S::BN * kChunks / S::kThreads;
        Pack<T> ra[kRegA], rb[kRegB];
        Operands set;
        const int whole = a.ld >= kPack<T> && b.ld >= kPack<T> ? steps - 1 : 0;
        auto fetch_step = [&](int t) {
            const int64_t k0 = (int64_t)t * kStep<T>;
            if (t < whole) {
                fetch<T, AKC, S::BM, S::kWaves, true>(a, k0, ra);
                fetch<T, BKC, S::BN, S::kWaves, true>(b, k0, rb);
            } else {
                fetch<T, AKC, S::BM, S::kWaves, false>(a, k0, ra);
                fetch<T, BKC, S::BN, S::kWaves, false>(b, k0, rb);
            }
        };
        auto put_step = [&](LdsByte *to) {
            put<T, AKC, S::BM, S::kWaves>(to, ra);
            put<T, BKC, S::BN, S::kWaves>(to + kA, rb);
        };
        if (steps > 0) {
            fetch_step(0);
            put_step(lds.at[0]);
        }
        __syncthreads();
        for (int t = 0; t < steps; t += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (t + u < steps) {
                    const bool more = t + u + 1 < steps;
                    if (more) fetch_step(t + u + 1);
                    read_step(lds.at[u], set);
                    multiply_step(set);
                    if (more) put_step(lds.at[1 - u]);
                    __syncthreads();
                }
            }
        }
    }
    // The outputs go through LDS (the stages, read out by now) so that a store
    // covers whole rows of the tile: a lane holds 4 columns of one row, and 32
    // rows to a store would reach the L2 as 16-byte pieces.  Chunk c of row r
    // stands at c ^ r.
    constexpr int kRow = S::BN * (int)sizeof(OUT), kRowChunks = kRow / 16;
    constexpr int kStageRows = S::kStageBytes / kRow / 32 * 32;
    static_assert(kStages * kStageRows >= S::BM, "the stages hold the tile");
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));                 // addresses of the stores are not kept through the loop
    const int lane = thread & (kWave - 1);
#pragma unroll
    for (int wr = 0; wr < S::WR; ++wr) {             // the stage is known at compile time
        if (wave / S::WC != wr) continue;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r0 = (wr * MI + i) * 32, r = r0 + (lane & 31);
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int byte = (n0 + j * 32 + q * 8 + (lane >> 5) * 4) * (int)sizeof(OUT);
                    struct alignas(4 * sizeof(OUT)) Four {
                        OUT v[4];
                    } o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o.v[e] = (OUT)acc[i][j][q * 4 + e];
                    LdsByte *p = lds.at[r0 / kStageRows] + r % kStageRows * kRow +
                                 (((byte >> 4) ^ (r & (kRowChunks - 1))) << 4) + (byte & 15);
                    if constexpr (sizeof(OUT) == 4) lds_store(p, o);
                    else *(__attribute__((address_space(3))) i32x2 *)p = __builtin_bit_cast(i32x2, o);
                }
        }
    }
    __syncthreads();
    constexpr int kRowsPerPass = S::kThreads / kRowChunks;
    const int chunk = thread % kRowChunks, c = chunk * kPack<OUT>;
#pragma unroll
    for (int r0 = 0; r0 < S::BM; r0 += kRowsPerPass) {
        const int r = r0 + thread / kRowChunks;
        const auto o = lds_load<Pack<OUT>>(lds.at[r0 / kStageRows] + r % kStageRows * kRow +
                                           ((chunk ^ (r & (kRowChunks - 1))) << 4));
        if (r >= rows) continue;
        if (stream) store_pack_stream(out + r * ldo + c, o, cols - c);
        else store_pack(out + r * ldo + c, o, cols - c);
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

// Blocks are dealt to the 8 XCDs in turn: give each XCD a run of consecutive
// tiles, whose operands then meet in one L2.
__device__ inline int64_t xcd_order(int64_t id, int64_t total) {
    const int64_t per = total / 8, extra = total % 8, x = id % 8, at = id / 8;
    return x * per + (x < extra ? x : extra) + at;
}

// The same for tiles that are to start in their order (dw's, longest segments
// first): groups of 8 consecutive tiles to an XCD, every other round of groups
// backwards, the last tiles one by one.  8 tiles to a segment (65,536 rows in
// 200, 512 x 1024 bf16) 133 -> 111 us, 16 tiles 166 -> 164, 32 tiles 291 -> 284;
// 64 tiles 262 both ways, 128 tiles 1001 -> 1013 us, so up to 32.  Groups of 32
// gain more for even segments (338 -> 311 against 329 us) but leave XCDs idle
// for uneven ones (398 -> 476 against 395 us).
__device__ inline int64_t xcd_groups(int64_t id, int64_t total) {
    const int64_t round = id / 64 * 64, in = id % 64, x = in % 8;
    if (round + 64 > total) return id;
    return round + (round & 64 ? 7 - x : x) * 8 + in / 8;
}

// Tiles of the runs [v0, v1), each cut into pieces of `len` rows and `cols`
// tiles to a piece: the piece and column tile of tile number `id`, numbered
// so that each XCD gets a run of them; run < 0: there are fewer tiles.  `most`
// tiles are the most that offsets in order can have; tiles beyond them, of
// offsets that decrease, are left out.  Every wave finds its tile by itself:
// 64 runs at a time, a scan of their pieces.
struct RowTile {
    int64_t run, row, end, piece, col;
};

__device__ inline int64_t pieces_of(const SegmentArgs &a, int64_t v, int64_t v1, int64_t len, int64_t *lo, int64_t *hi) {
    *lo = v < v1 ? run_bound(a, v) : 0;
    *hi = v < v1 ? run_bound(a, v + 1) : 0;
    return *hi > *lo ? (uint32_t)(*hi - *lo + len - 1) / (uint32_t)len : 0;
}

__device__ inline int64_t wave_inclusive(int64_t v) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int64_t up = __shfl_up(v, o, kWave);
        if (lane >= o) v += up;
    }
    return v;
}

// Pieces of the runs [v0, v1) together.
__device__ inline int64_t count_pieces(const SegmentArgs &a, int64_t v0, int64_t v1, int64_t len) {
    int64_t sum = 0, lo, hi;
    for (; v0 < v1; v0 += kWave) sum += pieces_of(a, v0 + (threadIdx.x & (kWave - 1)), v1, len, &lo, &hi);
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    return uniform(sum);
}

__device__ inline RowTile find_tile(const SegmentArgs &a, int64_t v0, int64_t v1, int64_t len, int64_t cols, int64_t id,
                                   int64_t most) {
    const int lane = threadIdx.x & (kWave - 1);
    RowTile t = {-1, 0, 0, 0, 0};
    int64_t lo, hi, mine = pieces_of(a, v0 + lane, v1, len, &lo, &hi), incl = wave_inclusive(mine);
    const int64_t first = __shfl(incl, kWave - 1, kWave);
    const int64_t count = uniform(v1 - v0 <= kWave ? first : first + count_pieces(a, v0 + kWave, v1, len));
    const int64_t total = min(count * cols, most);
    if (id >= total) return t;
    const int64_t at = xcd_order(id, total);
    t.piece = at / cols;
    t.col = at % cols;
    int64_t piece = t.piece;
    for (;;) {
        const uint64_t past = __ballot(incl > piece);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            t.run = uniform(v0 + l);
            t.row = uniform(__shfl(lo, l, kWave) + (piece - __shfl(incl - mine, l, kWave)) * len);
            t.end = uniform(__shfl(hi, l, kWave));
            return t;
        }
        piece -= __shfl(incl, kWave - 1, kWave);
        v0 += kWave;
        if (v0 >= v1) return t;
        mine = pieces_of(a, v0 + lane, v1, len, &lo, &hi);
        incl = wave_inclusive(mine);
    }
}

// The same for many runs, where counting the pieces of all of them in every
// wave would cost the square of their number.  Run v, from row lo, owns the
// slots from lo / LEN + v on to the next run's: at least as many as it has
// pieces, since ceil(n / LEN) <= floor((lo + n) / LEN) - floor(lo / LEN) + 1.
// The slots' run is found by a search that looks at 64 runs at a time; the
// slots that a run does not need hold no rows.  From 127 segments on, more than
// two scans (segments of uneven lengths, 64 x 64 bf16): 40 rows to a segment, 126
// segments 8.5 us both ways, 190 9.3 -> 9.0, 512 23 -> 12, 2000 147 -> 29, 65,536
// segments 224 -> 2.2 ms; 400 rows to a segment, 126 11.9 -> 12.6 us, 190 17.7 ->
// 15.0, 512 79 -> 50, 2000 591 -> 168.
constexpr int kScannedSegments = 126;

template <int LEN>
__device__ inline RowTile find_slot(const SegmentArgs &a, int64_t cols, int64_t id, int64_t total) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t at = xcd_order(id, total);
    RowTile t;
    t.piece = at / cols;
    t.col = at % cols;
    int64_t v = 0, n = a.E + 2;                      // the run is one of n from v on
    while (n > 1) {
        const int64_t step = (n + kWave - 1) / kWave, to = lane * step;
        const bool from = lane == 0 || (to < n && run_bound(a, v + to) / LEN + v + to <= t.piece);
        const int64_t past = (kWave - 1 - __builtin_clzll(__ballot(from))) * step;
        v += past;
        n = min(step, n - past);
    }
    const int64_t lo = run_bound(a, v);
    t.run = uniform(v);
    t.row = uniform(lo + (t.piece - lo / LEN - v) * LEN);
    t.end = uniform(run_bound(a, v + 1));
    return t;
}

template <typename T, typename S, bool TRANSPOSED, bool DIRECT>
__global__ __launch_bounds__(S::kThreads, 2) void segment_kernel(SegmentArgs a, int64_t col_tiles, int64_t total,
                                                                bool stream) {
    SEGMENT_STAGES(lds, S::kStageBytes);
    const int64_t K = TRANSPOSED ? a.O : a.I, N = TRANSPOSED ? a.I : a.O;
    const T *in = (const T *)(TRANSPOSED ? a.dy : a.x), *w = (const T *)a.w;
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        RowTile rt;
        if (a.E > kScannedSegments) {
            rt = find_slot<S::BM>(a, col_tiles, id, total);
            if (rt.row < 0 || rt.row >= rt.end) continue;
        } else {
            rt = find_tile(a, 0, a.E + 2, S::BM, col_tiles, id, total);
            if (rt.run < 0) return;
        }
        const int64_t run = uniform(rt.run), row = uniform(rt.row), n0 = rt.col * S::BN;
        T *out = (T *)a.y + row * N + n0;
        const int64_t rows = uniform(rt.end) - row;
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
        tile_product<T, T, S, true, TRANSPOSED, DIRECT>(lds, A, B, K, out, N, rows, N - n0, stream);
    }
}

// Segment whose length is the `rank`-th largest (ties by number), for up to 64.
__device__ inline int64_t segment_by_length(const SegmentArgs &a, int rank) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t len = lane < a.E ? run_bound(a, lane + 2) - run_bound(a, lane + 1) : INT64_MIN;
    int before = 0;
    for (int e = 0; e < (int)a.E; ++e) {
        const int64_t other = __shfl(len, e, kWave);
        before += other > len || (other == len && e < lane);
    }
    return uniform((int)__ffsll((unsigned long long)__ballot(lane < a.E && before == rank)) - 1);
}

// dw.  chunk == 0: tile (segment, tile of [I, O]) over all rows of the
// segment; of up to 64 segments the longest start first.  chunk > 0: tile (chunk of a
// segment's rows, tile of [I, O]) into fp32 partial sums, one [I, O] for each
// chunk in the order of the segments.
template <typename T, typename OUT, typename S, bool DIRECT>
__global__ __launch_bounds__(S::kThreads, 2) void segment_dw_kernel(SegmentArgs a, OUT *dst, int64_t row_tiles,
                                                                 int64_t col_tiles, int64_t chunk, int64_t total,
                                                                 bool stream) {
    SEGMENT_STAGES(lds, S::kStageBytes);
    for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
        const int64_t tiles = row_tiles * col_tiles;
        int64_t t, at, row, end;
        if (chunk) {
            const RowTile rt = find_tile(a, 1, a.E + 1, chunk, tiles, id, total);
            if (rt.run < 0) return;
            t = rt.piece;
            at = rt.col;
            row = uniform(rt.row);
            end = min(uniform(rt.end), row + chunk);
        } else {
            const int64_t tile = tiles <= 32 ? xcd_groups(id, total) : id;
            t = tile / tiles;
            at = tile % tiles;
            if (a.E <= kWave) t = max(int64_t(0), segment_by_length(a, (int)t));
            row = run_bound(a, t + 1);
            end = max(row, run_bound(a, t + 2));
        }
        const int64_t m0 = at / col_tiles * S::BM, n0 = at % col_tiles * S::BN;
        Operand<T> A, B;
        A.ptr = (const T *)a.x + row * a.I + m0;
        A.ld = a.I;
        A.outer = end - row;
        A.inner = a.I - m0;
        A.end = (const T *)a.x + a.R * a.I;
        B.ptr = (const T *)a.dy + row * a.O + n0;
        B.ld = a.O;
        B.outer = end - row;
        B.inner = a.O - n0;
        B.end = (const T *)a.dy + a.R * a.O;
        __syncthreads();
        tile_product<T, OUT, S, false, false, DIRECT>(lds, A, B, end - row, dst + (t * a.I + m0) * a.O + n0, a.O,
                                                      a.I - m0, a.O - n0, stream);
    }
}

constexpr int kFoldThreads = 256;

// Adds a segment's partial sums in the order of its chunks.
template <typename T>
__global__ __launch_bounds__(kFoldThreads) void segment_fold_kernel(SegmentArgs a, int64_t chunk,
                                                                    int64_t chunks) {
    const int64_t n = a.I * a.O;
    for (int64_t e = blockIdx.y; e < a.E; e += gridDim.y) {
        const int64_t first = min(chunks, count_pieces(a, 1, e + 1, chunk));
        const int64_t parts = min(chunks - first, count_pieces(a, e + 1, e + 2, chunk));
        const float *from = a.partial + first * n;
        for (int64_t i = (int64_t)blockIdx.x * kFoldThreads + threadIdx.x; i < n;
             i += (int64_t)gridDim.x * kFoldThreads) {
            float t = 0.0f;
#pragma unroll 8
            for (int64_t p = 0; p < parts; ++p) t += from[p * n + i];
            ((T *)a.y)[e * n + i] = (T)t;
        }
    }
}

int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

constexpr int64_t kMaxBlocks = 1 << 20;
constexpr int64_t kUnits = 256;                      // compute units

// Non-temporal stores where a call moves more than half of the 256 MB Infinity
// Cache, so that the operands that other tiles read again stay there.  65,536
// rows, 1024 x 2048 bf16, calls of both kinds and directions in turn: 32 segments
// y 308 -> 302, dx 292 -> 278 us; one segment 296 -> 289 and 274 -> 267, with 256
// summed elements 130 -> 122 and 118 -> 110.  In a loop of one call, whose
// outputs would push out its own operands, one segment's y 319 -> 269 to 293 and
// 143 -> 110 to 136 us.
constexpr int64_t kStreamBytes = int64_t(128) << 20;

template <typename T>
bool streams(const SegmentArgs &a) {
    return (a.R * (a.I + a.O) + a.E * a.I * a.O) * (int64_t)sizeof(T) > kStreamBytes;
}

// The copy into LDS needs rows of whole 16-byte groups, from a 16-byte
// address, and 32-bit offsets within a tile's rows.
bool direct_rows(const void *p, int64_t width, int size) {
    return (uintptr_t)p % 16 == 0 && width * size % 16 == 0 && width * size * 320 < (int64_t(1) << 31);
}

// 256 x 256 tiles when there are enough of them to fill the chip.
bool large_tiles(int64_t tiles, int size, bool direct) { return direct && size == 2 && tiles >= 2 * kUnits; }

// dw: whole segments when their tiles fill the chip twice or there are few
// rows (then one long segment costs less than the partial sums); else chunks of
// rows, about two tiles of work for each compute unit (150,001 fp32 rows of 7
// segments, 128 x 256: 110 us with the sums' 11; with four 131 and 19 us) and at
// least 256 elements of the summed index, so that unequal segments cost no
// balance.
struct DwShape {
    bool large;
    int64_t row_tiles, col_tiles;
    int64_t chunk, chunks;       // rows of a chunk (0: whole segments) and the most chunks there can be
};

DwShape dw_shape(int64_t R, int64_t E, int64_t I, int64_t O, int size, bool direct) {
    DwShape d;
    d.large = large_tiles(E * tiles_of(I, 256) * tiles_of(O, 256), size, direct);
    const int tile = d.large ? 256 : 128;
    d.row_tiles = tiles_of(I, tile);
    d.col_tiles = tiles_of(O, tile);
    const int64_t tiles = d.row_tiles * d.col_tiles, want = std::max<int64_t>(1, 2 * kUnits / tiles);
    d.chunk = d.chunks = 0;
    if (E * tiles >= 2 * kUnits || R <= 4096) return d;
    d.chunk = std::max<int64_t>(256, (R + want - 1) / want);
    d.chunk = (d.chunk + 31) / 32 * 32;
    d.chunks = R / d.chunk + E;
    return d;
}

template <typename T, typename S, bool DIRECT>
hipError_t segment_launch(const SegmentArgs &a, bool transposed, hipStream_t s) {
    // each run adds at most one partial tile
    const int64_t row_tiles = a.R / S::BM + a.E + 2, col_tiles = tiles_of(transposed ? a.I : a.O, S::BN);
    const int64_t total = row_tiles * col_tiles;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    const bool stream = streams<T>(a);
    if (transposed) segment_kernel<T, S, true, DIRECT><<<blocks, S::kThreads, 0, s>>>(a, col_tiles, total, stream);
    else segment_kernel<T, S, false, DIRECT><<<blocks, S::kThreads, 0, s>>>(a, col_tiles, total, stream);
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
    const int64_t total = (d.chunk ? d.chunks : a.E) * d.row_tiles * d.col_tiles;
    const unsigned blocks = (unsigned)std::min(total, kMaxBlocks);
    const bool stream = d.chunk == 0 && streams<T>(a);       // partial sums are read again at once
    if constexpr (sizeof(T) == 2 && __is_same(T, OUT)) {       // large tiles take whole segments
        if (d.large) {
            segment_dw_kernel<T, OUT, Large, true><<<blocks, Large::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                     d.chunk, total, stream);
            return hipGetLastError();
        }
    }
    if (direct)
        segment_dw_kernel<T, OUT, Medium, true><<<blocks, Medium::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                   d.chunk, total, stream);
    else
        segment_dw_kernel<T, OUT, Medium, false><<<blocks, Medium::kThreads, 0, s>>>(a, dst, d.row_tiles, d.col_tiles,
                                                                                    d.chunk, total, stream);
    return hipGetLastError();
}

template <typename T>
hipError_t segment_dw(const SegmentArgs &a, hipStream_t s) {
    const bool direct = direct_rows(a.x, a.I, sizeof(T)) && direct_rows(a.dy, a.O, sizeof(T));
    const DwShape d = dw_shape(a.R, a.E, a.I, a.O, sizeof(T), direct);
    if (d.chunk == 0) return segment_dw_launch<T, T>(a, (T *)a.y, d, direct, s);
    if (const hipError_t e = segment_dw_launch<T, float>(a, a.partial, d, direct, s)) return e;
    const int64_t n = a.I * a.O;
    const dim3 grid((unsigned)std::min<int64_t>((n + kFoldThreads - 1) / kFoldThreads, 1 << 16),
                    (unsigned)std::min<int64_t>(a.E, 1 << 14));
    segment_fold_kernel<T><<<grid, kFoldThreads, 0, s>>>(a, d.chunk, d.chunks);
    return hipGetLastError();
}

}  // namespace

int64_t segment_workspace_floats(int64_t R, int64_t E, int64_t I, int64_t O, int type) {
    // the addresses are not known here: what either way of staging needs
    int64_t chunks = 0;
    for (const bool direct : {false, true})
        chunks = std::max(chunks, dw_shape(R, E, I, O, type == SPMM_F32 ? 4 : 2, direct).chunks);
    return chunks * I * O;
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
