// Matrix products of tiles on the matrix cores, for rows of fp32, bf16 or fp16:
// a block's sums of one tile, and their way out through LDS.  The segment product
// and the classifier's loss are made of it.
//
// A tile is computed in steps of 64 bytes of the summed index (32 16-bit or 16
// fp32 elements).  Both operands' steps are copied straight into LDS in the
// orientation they have in memory, four steps ahead of the matrix instructions;
// operands whose rows are the summed index are turned by the transposing LDS read
// (16-bit) or read element by element (fp32).
#pragma once

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
// of row k at c ^ 2 (k & 3) (B = 64, two rows to the banks: c ^ 2 (k / 2 & 1)), so
// that the four rows a 16-lane transposing read touches lie in different banks.
// fp32: 16 rows of 4 B bytes, as they are.

template <int B>
__device__ inline int turned_piece(int k) {
    static_assert(B >= 64);
    return B >= 128 ? (k & 3) << 1 : (k >> 1 & 1) << 1;
}

template <typename T, bool KC, int B>
__device__ inline int chunk_offset(int outer, int chunk) {
    if constexpr (KC) return outer * kStepBytes + ((chunk ^ (outer >> 2 & 3)) << 4);
    else if constexpr (sizeof(T) == 4) return outer * B * 4 + (chunk << 4);
    else return outer * B * 2 + (((chunk >> 1) ^ turned_piece<B>(outer)) << 5) + ((chunk & 1) << 4);
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
    const int *rows = nullptr;      // KC: tile row r is row rows[r] from ptr (GATHER)
};

// Copies an operand's steps straight into LDS, 16 bytes per lane: for rows
// that start on 16 bytes and are multiples of them.  A lane's place in the
// step is fixed by its number, so the swizzle is applied to what it reads.
// What lies behind the summed range reads as zero (the lane points behind the
// buffer); tile rows (KC) and columns (KS) that do not exist read what
// follows in the same array, or zero behind its end: they only reach outputs
// that are not stored.
// GATHER (KC): rows by their list, within 2^31 - 1 bytes of ptr; the rows behind
// the last one repeat it.
template <typename T, bool KC, int B, int WAVES, bool GATHER = false>
struct Copy {
    static_assert(KC || !GATHER);
    static constexpr int kCopies = B * kStepBytes / 1024 / WAVES;
    static constexpr int kRowsPerCopy = KC ? 1024 / kStepBytes * WAVES : 1024 * WAVES / (B * (int)sizeof(T));

    const char *base;
    int64_t bytes;          // from base to the end of the array
    int64_t step_bytes;
    uint32_t at, next_copy; // byte offset of the lane's chunk of copy 0, and from one copy to the next
    int first;              // the lane's first summed element of copy 0 within a step
    int left;               // summed elements from the next step on
    uint32_t listed[GATHER ? kCopies : 1];

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
            if constexpr (GATHER) {
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int64_t r = min(int64_t(row + i * kRowsPerCopy), o.outer - 1);
                    listed[i] = (uint32_t)o.rows[r] * row_bytes + chunk * 16;
                }
            }
        } else {
            constexpr int kRow = B * (int)sizeof(T);
            const int k = byte / kRow;
            int chunk = byte % kRow / 16;
            if constexpr (sizeof(T) == 2) chunk = (((chunk >> 1) ^ turned_piece<B>(k)) << 1) | (chunk & 1);
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
            uint32_t from = at + i * next_copy;
            if constexpr (GATHER) from = listed[i];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(lds + (i * WAVES + wave) * 1024), 16,
                in ? from : 0x80000000u, 0, 0, 0);
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
template <typename T, bool KC, int B, int WAVES, bool WHOLE, bool GATHER = false>
__device__ inline void fetch(const Operand<T> &o, int64_t k0, Pack<T> (&r)[B * kChunks / (WAVES * kWave)]) {
    constexpr int kPerRow = KC ? kStepBytes / 16 : B * (int)sizeof(T) / 16;
#pragma unroll
    for (int i = 0; i < B * kChunks / (WAVES * kWave); ++i) {
        const int idx = threadIdx.x + i * WAVES * kWave, row = idx / kPerRow, c = idx % kPerRow * kPack<T>;
        if constexpr (WHOLE) {
            int64_t out = KC ? min(int64_t(row), o.outer - 1) : k0 + row;
            const int64_t in = KC ? k0 + c : min(int64_t(c), o.inner - 1);
            if constexpr (GATHER) out = o.rows[out];
            r[i] = load_pack(o.ptr + out * o.ld + in);
        } else {
            int64_t out = KC ? row : k0 + row;
            const int64_t in = KC ? k0 + c : c, n = out < o.outer ? o.inner - in : 0;
            if constexpr (GATHER) out = o.rows[min(out, o.outer - 1)];
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
                at[i] = k * B * 2 + ((piece ^ turned_piece<B>(k)) << 5) + ((l & 3) << 3);
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

#define TILE_STAGES(name, bytes)                                                                 \
    __shared__ __attribute__((aligned(1024))) char name##0[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##1[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##2[bytes];                                  \
    __shared__ __attribute__((aligned(1024))) char name##3[bytes];                                  \
    const Stages name = {{(LdsByte *)name##0, (LdsByte *)name##1, (LdsByte *)name##2, (LdsByte *)name##3}}

// The sums of a wave's part of a tile: rows 32 i and columns 32 j from the
// wave's corner, laid out as multiply() leaves them.
template <typename S>
struct Sums {
    f32x16 at[S::MI][S::NI];
};

// out += A . B over K summed elements; LDS is free for other use afterwards.
// GATHER: A's rows by their list.
template <typename T, typename S, bool AKC, bool BKC, bool DIRECT, bool GATHER = false>
__device__ inline void tile_sums(const Stages &lds, const Operand<T> &a, const Operand<T> &b, int64_t K, Sums<S> &out) {
    f32x16 (&acc)[S::MI][S::NI] = out.at;
    constexpr int MI = S::MI, NI = S::NI, kA = S::BM * kStepBytes;
    const int wave = uniform((int)threadIdx.x / kWave);
    const int m0 = wave / S::WC * (MI * 32), n0 = wave % S::WC * (NI * 32);
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
        Copy<T, AKC, S::BM, S::kWaves, GATHER> ca(a, wave);
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
                fetch<T, AKC, S::BM, S::kWaves, true, GATHER>(a, k0, ra);
                fetch<T, BKC, S::BN, S::kWaves, true>(b, k0, rb);
            } else {
                fetch<T, AKC, S::BM, S::kWaves, false, GATHER>(a, k0, ra);
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
}

// out[0..rows) x [0..cols) of a tile = the sums.  The outputs go through LDS (the
// stages, read out by now) so that a store covers whole rows of the tile: a lane
// holds 4 columns of one row, and 32 rows to a store would reach the L2 as
// 16-byte pieces.  Chunk c of row r stands at c ^ r.  `list`: row r goes to row
// list[r] of out.
template <typename OUT, typename S, bool LISTED = false>
__device__ inline void tile_store(const Stages &lds, const Sums<S> &sums, OUT *out, int64_t ldo, int64_t rows,
                                  int64_t cols, bool stream, const int *list = nullptr) {
    const f32x16 (&acc)[S::MI][S::NI] = sums.at;
    constexpr int MI = S::MI, NI = S::NI;
    const int wave = uniform((int)threadIdx.x / kWave);
    const int n0 = wave % S::WC * (NI * 32);
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
        const int64_t to = LISTED ? list[r] : r;
        if (stream) store_pack_stream(out + to * ldo + c, o, cols - c);
        else store_pack(out + to * ldo + c, o, cols - c);
    }
}

// out[0..rows) x [0..cols) of a tile = the sums (ADD: added to out) in fp32, straight from
// the registers: the stages do not hold a large tile of fp32.
template <typename S, bool ADD>
__device__ inline void tile_store_fp32(const Sums<S> &sums, float *out, int64_t ldo, int64_t rows, int64_t cols) {
    const f32x16 (&acc)[S::MI][S::NI] = sums.at;
    const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
    const int m0 = wave / S::WC * (S::MI * 32), n0 = wave % S::WC * (S::NI * 32);
#pragma unroll
    for (int i = 0; i < S::MI; ++i) {
        const int r = m0 + i * 32 + (lane & 31);
        if (r >= rows) continue;
#pragma unroll
        for (int j = 0; j < S::NI; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = n0 + j * 32 + q * 8 + (lane >> 5) * 4;
                float *p = out + r * ldo + c;
                Pack<float> v;
                if constexpr (ADD) v = load_pack(p, cols - c);
#pragma unroll
                for (int e = 0; e < 4; ++e) v.v[e] = ADD ? v.v[e] + acc[i][j][q * 4 + e] : acc[i][j][q * 4 + e];
                store_pack(p, v, cols - c);
            }
    }
}

// out[0..rows) x [0..cols) of a tile = A . B over K summed elements.
template <typename T, typename OUT, typename S, bool AKC, bool BKC, bool DIRECT>
__device__ inline void tile_product(const Stages &lds, const Operand<T> &a, const Operand<T> &b, int64_t K, OUT *out,
                                    int64_t ldo, int64_t rows, int64_t cols, bool stream) {
    Sums<S> sums = {};
    tile_sums<T, S, AKC, BKC, DIRECT>(lds, a, b, K, sums);
    tile_store<OUT, S>(lds, sums, out, ldo, rows, cols, stream);
}

}  // namespace

}  // namespace gspmm
