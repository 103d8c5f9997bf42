// Attention among the rows of each segment, and its gradients.  For a row i of
// segment s and a head h, over the keys j of s (causal: j <= i + m - n for the
// n rows and m keys of s, both counted from its start):
//
//   out_i = sum_j p_ij v_j,   p_ij = exp(scale q_i.k_j) / sum_j exp(scale q_i.k_j)
//
//   dv_j = sum_i p_ij dout_i            ds_ij = p_ij (dout_i.v_j - dout_i.out_i)
//   dq_i = scale sum_j ds_ij k_j        dk_j  = scale sum_i ds_ij q_i
//
// One pass over the keys with the running maximum and sum of the softmax; the
// scores never leave the registers.  The G = H / Hk query heads of a key head
// are packed into its rows (packed row i G + g), so a step with one new row per
// sequence fills tiles with its heads, keys are read once for all of a group,
// and the sums over a group's heads in dk and dv are sums over rows.
//
// A wave owns 32 packed rows (32 keys in dk and dv) and walks tiles of keys
// (rows) in LDS.  Scores are computed with the tile's rows in the registers and
// the wave's own in the lanes, so a row's maximum and sum are in-lane plus one
// exchange of the two half waves, and the products of the second stage take the
// probabilities from the registers they are in: the summed index may stand in
// any order, so the turned LDS reads of v (k, q, dout) follow the order that the
// matrix instruction left.  Tiles are copied into LDS ahead of their use, 16
// bytes per lane, chunks placed so that both ways of reading meet no bank twice.
//
// Sums and statistics are fp32.  Probabilities and ds are rounded to the rows'
// type where they enter a matrix instruction (16-bit types).  fp16 has 2^-14 to 2^16
// for them, so they are held times powers of two that are taken out of the sums
// again: p times 2^12 (forward: the running maximum's, so that 60,000 keys of 2^-22 of
// the largest weight still add up), and in the gradients ds, a share of 1 / keys of
// dout.v, times what brings a row's largest so far to 2^11 or more (dq, HeldGradients) or
// what bounds a key's to 2^15 (dk, KeySums::hold).
//
// dk and dv are computed apart from dq, which takes two products more than one
// kernel for all three would: added up in dq's order or dk's, one of them would need
// atomics, whose order changes results.
//
// Bound by the matrix cores and the exponentials between them, each about as long;
// medians of the kernels alone over 20 calls under the profiler, 128-element heads, causal,
// bf16: 12,001 rows in 5 segments, 32 heads over 8, 430 us (350 to 375 us a call in loops of
// several hundred without it, 830 to 890 TFLOP/s; matrix cores 40%, vector units 39% busy, no
// LDS bank conflicts).  8,192 rows in 3, 16 over 4: forward 155 us (655), dq 183 (828 over its
// three products), dk and dv 338 + 27 for the parts' sum (598 over four; one wave to a SIMD,
// 28% and 26% busy, a quarter of the units idle at its end).  One row each against 100,003
// keys in 32 segments: 89 + 8 us, 410 MB at 4.2 TB/s.  4,096 graphs of 24 rows, 4 heads of
// 32, fp32: 81, 106 and 134 us, fp32 matrix instructions 33 to 41% busy on 32 x 32 tiles
// of which the graphs fill half.  All by segments of like length: the launches go by the
// mean (attention.hip).
#pragma once

#include "tile_product.h"

namespace gspmm {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// ---- exact division by a number fixed on the host, for n < 2^31 ----

__device__ inline int quotient(const Divisor &d, int n) {
    return (int)(((uint64_t)(uint32_t)n * d.magic) >> d.shift);
}

// ---- LDS layout of a tile: rows of kPitch bytes, a power of two ----
//
// Chunk c of row r stands at c ^ place(r).  16 lanes that read one chunk of 16
// rows, and 32 lanes that turn 4 rows of 64 bytes, cover the 64 banks once.
template <typename T, int DP>
struct Tile {
    static constexpr int kPitch = DP * (int)sizeof(T) <= 64 ? 64 : DP * (int)sizeof(T) <= 128 ? 128
                                  : DP * (int)sizeof(T) <= 256 ? 256 : 512;
    static constexpr int kChunks = kPitch / 16;
    static constexpr int kDrop = kChunks >= 16 ? 0 : kChunks == 8 ? 1 : 2;
    static constexpr int kSteps = DP * (int)sizeof(T) / 32;      // matrix steps along a row
    static constexpr int kBlocks = DP / 32;                      // 32-element blocks of a row
    static constexpr int kGroups = 16 / kPack<T>;                // matrix steps along 32 rows

    static __device__ inline int place(int r) { return ((r & 3) >> kDrop) << 2 | (r >> 2 & 3); }
};

// The lane's operand of matrix step ks: row block * 32 + lane % 32.
template <typename T, int DP>
struct RowReader {
    using L = Tile<T, DP>;
    int at;

    __device__ inline RowReader() {
        const int lane = threadIdx.x & (kWave - 1), r = lane & 31;
        at = r * L::kPitch + (((lane >> 5) ^ L::place(r)) << 4);
    }

    __device__ inline Pack<T> read(LdsByte *tile, int block, int ks) const {
        return lds_load<Pack<T>>(tile + ((at ^ (ks << 5)) + block * 32 * L::kPitch));
    }
};

// The same of the tile turned: element d * 32 + lane % 32 of the rows that the
// registers group * kPack .. of multiply() stand for in the lane's half.
template <typename T, int DP>
struct TurnedReader {
    using L = Tile<T, DP>;
    int at;

    __device__ inline TurnedReader() {
        const int lane = threadIdx.x & (kWave - 1), half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            // lane l of 16 points at 4 elements of row l / 4 and receives
            // element l of the rows 0..3
            const int l = lane & 15, r = 4 * half + (l >> 2);
            const int chunk = (lane >> 4 & 1) * 2 + (l >> 1 & 1);
            at = r * L::kPitch + ((chunk ^ L::place(r)) << 4) + (l & 1) * 8;
        } else {
            at = 4 * half * L::kPitch + (((lane & 31) >> 2 ^ half) << 4) + (lane & 3) * 4;
        }
    }

    __device__ inline Pack<T> read(LdsByte *tile, int block, int group, int d) const {
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) i16x4 LdsFour;
            struct {
                i16x4 lo, hi;
            } both;
            const int row = (block * 32 + group * 16) * L::kPitch;
            both.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsFour *)(tile + ((at ^ (d << 6)) + row)));
            both.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (LdsFour *)(tile + ((at ^ (d << 6) ^ 32) + (row + 8 * L::kPitch))));
            return __builtin_bit_cast(Pack<T>, both);
        } else {
            Pack<T> r;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int place = (d * 8) ^ ((j >> L::kDrop) << 2) ^ (2 * group & 3);
                const int row = (block * 32 + 8 * group + j) * L::kPitch;
                r.v[j] = *(__attribute__((address_space(3))) float *)(tile + ((at ^ (place << 4)) + row));
            }
            return r;
        }
    }
};

// ---- rows of a tile in memory ----

// Consecutive rows of one head.
template <typename T>
struct KeyRows {
    const T *base;
    int64_t ld;
    int left;           // rows that exist

    __device__ inline int64_t at(int r) const { return r * ld; }
};

// Consecutive packed rows of one key head, from packed row m0 of a segment;
// base: row m0 / G, the group's first head.
template <typename T>
struct PackedRows {
    const T *base;
    int64_t ld;
    int left, m0, i0, D;
    Divisor G;

    __device__ inline int64_t at(int r) const {
        const int m = m0 + r, i = quotient(G, m);
        return (i - i0) * ld + (m - i * G.d) * D;
    }
};

// Fills ROWS rows of a tile, zeros where a row or an element does not exist.
// DIRECT: copied straight into LDS from the offsets that aim() left; else through
// registers, load() ahead of the use of what put() overwrites.
template <typename T, int DP, int ROWS, int WAVES, bool DIRECT>
struct Fill {
    using L = Tile<T, DP>;
    static constexpr int kCopies = ROWS * L::kPitch / 1024 / WAVES;
    static constexpr uint32_t kNowhere = 0x80000000u;    // behind 2^31 - 1 bytes the copy writes zeros
    Pack<T> r[DIRECT ? 1 : kCopies];
    uint32_t off[DIRECT ? kCopies : 1];

    static __device__ inline int row_of(int i, int wave) {
        return ((i * WAVES + wave) * 1024 + (threadIdx.x & (kWave - 1)) * 16) / L::kPitch;
    }
    static __device__ inline int element_of(int i, int wave) {
        const int byte = (i * WAVES + wave) * 1024 + (threadIdx.x & (kWave - 1)) * 16;
        return ((byte % L::kPitch / 16) ^ L::place(byte / L::kPitch)) * kPack<T>;
    }

    template <typename Rows>
    __device__ inline void aim(const Rows &rows, int D, int wave) {
        if constexpr (DIRECT) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int e = element_of(i, wave);
                off[i] = e < D ? (uint32_t)(rows.at(row_of(i, wave)) + e) * (uint32_t)sizeof(T) : kNowhere;
            }
        }
    }

    template <typename Rows>
    __device__ inline void load(LdsByte *lds, const Rows &rows, int D, int wave) {
        if constexpr (DIRECT) {
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)uniform((int64_t)rows.base), 0, 0x7fffffff,
                                                                0x00020000);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const uint32_t from = row_of(i, wave) < rows.left ? off[i] : kNowhere;
                LdsByte *to = lds + (i * WAVES + wave) * 1024;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 16, from, 0, 0,
                                                         0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int row = row_of(i, wave), e = element_of(i, wave);
                const bool in = row < rows.left;
                r[i] = load_pack(rows.base + (in ? rows.at(row) + e : 0), in ? D - e : 0);
            }
        }
    }

    __device__ inline void put(LdsByte *lds, int wave) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                lds_store(lds + ((i * WAVES + wave) * 1024 + (threadIdx.x & (kWave - 1)) * 16), r[i]);
        }
    }
};

// ---- the tiles of a call ----

// S segments between rows (each `scale` packed rows) as S + 2 runs: the rows
// before the first segment, the segments, the rows behind the last.
struct Runs {
    const int64_t *offsets;
    int S, rows, scale;

    __device__ inline Runs(const int64_t *o, int64_t s, int64_t r, int by)
        : offsets(o), S((int)s), rows((int)r), scale(by) {}

    __device__ inline int bound(int v) const {
        if (v <= 0) return 0;
        if (v > S + 1) return rows;
        const int64_t b = offsets[v - 1];
        return b < 0 ? 0 : b > rows ? rows : (int)b;
    }
};

// Run v, from packed row lo, owns the slots from lo / LEN + v on to the next
// run's: at least as many as it has tiles of LEN rows.  The slot's run is found
// by a search that looks at 64 runs at a time; a slot that its run does not need
// has tile >= tiles.
struct Slot {
    int run, row0;                // the run's first row
    int rows, packed;             // how many it has
    int tile, tiles;
};

template <int LEN>
__device__ inline Slot find(const Runs &a, int slot) {
    const int lane = threadIdx.x & (kWave - 1);
    int v = 0, n = a.S + 2;
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave, to = lane * step;
        const bool from = lane == 0 || (to < n && a.bound(v + to) * a.scale / LEN + v + to <= slot);
        const int past = (kWave - 1 - __builtin_clzll(__ballot(from))) * step;
        v += past;
        n = min(step, n - past);
    }
    // lanes 0 and 1 load both bounds at once
    const int bound = a.bound(v + (lane & 1));
    Slot s;
    s.run = uniform(v);
    s.row0 = __builtin_amdgcn_readlane(bound, 0);
    s.rows = max(0, __builtin_amdgcn_readlane(bound, 1) - s.row0);
    s.packed = s.rows * a.scale;
    s.tiles = (s.packed + LEN - 1) / LEN;
    s.tile = slot - s.row0 * a.scale / LEN - s.run;
    if (s.tile < 0 || s.tile > s.tiles) s.tile = s.tiles;
    return s;
}

__device__ inline float other_half(float v) { return __shfl_xor(v, 32, kWave); }

__device__ inline float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// Key of register i of a score block, from the block's first.
__device__ inline int register_row(int i) {
    return 8 * (i >> 2) + 4 * ((threadIdx.x & (kWave - 1)) >> 5) + (i & 3);
}

// Types that hold probabilities times 2^kHeldBits, and ds, in the products.
template <typename T>
constexpr bool kHolds = __is_same(T, _Float16);
template <typename T>
constexpr float kHeldBits = kHolds<T> ? 12.0f : 0.0f;

// By how many powers of two a forward weight may pass the maximum that it is taken
// against: what is held stays below 2^15 in fp16.
template <typename T>
constexpr float kGrowth = kHolds<T> ? 3.0f : 8.0f;

// ds of a lane's row, held times a power of two `by` where fp16 takes it.  By the
// running largest, like a softmax's maximum: from 2^15 on, which is below fp16's
// largest, it is brought to 2^11 to 2^12 and the sums so far follow, exactly.  What is
// smaller than the largest by up to 2^25 keeps its eleven bits.  Starts at 2^60: times
// the largest there can be (2^12 p, 128 products of 2^16 by 2^16, twice) it stays finite,
// and what does not reach 2^15 then has gradients below fp16's smallest number.  8,192
// causal rows, 16 heads of 128 over 4: dq 187 -> 204 us.
template <typename T>
struct HeldGradients {
    float by = kHolds<T> ? 0x1p60f : 1.0f;

    template <int BLOCKS>
    __device__ inline void follow(f32x16 &ds, f32x16 (&sums)[BLOCKS]) {
        if constexpr (kHolds<T>) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(ds[i]));
            // rare: the sums stay where the matrix instructions have them
            if (__builtin_expect(__any(most >= 0x1p15f), 0)) {
                most = fmaxf(most, other_half(most));
                // infinities (their row's gradients are infinite or NaN) leave `by` alone
                const int e = most >= 0x1p15f && most < INFINITY ? 12 - __builtin_amdgcn_frexp_expf(most) : 0;
                const float f = ldexpf(1.0f, e);
                by *= f;
                ds *= f;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) sums[b] *= f;
            }
        }
    }
};

template <int CTRL>
__device__ inline float most_of_lanes(float v) {
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf,
                                                                          false)));
}

// The largest v of the wave's lanes: within quads, quads of 8, halves of 16, then rows of
// 16 through scalar registers.
__device__ inline float wave_most(float v) {
    v = most_of_lanes<0x4E>(most_of_lanes<0xB1>(v));
    v = most_of_lanes<0x140>(most_of_lanes<0x141>(v));
    const int bits = __builtin_bit_cast(int, v);
    auto lane = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits, l)); };
    return fmaxf(fmaxf(lane(0), lane(16)), fmaxf(lane(32), lane(48)));
}

// The length of the lane's row, its halves in both half waves.
template <typename T, int STEPS>
__device__ inline float length_of(const Pack<T> (&r)[STEPS]) {
    float sum = 0.0f;
#pragma unroll
    for (int ks = 0; ks < STEPS; ++ks)
#pragma unroll
        for (int e = 0; e < kPack<T>; ++e) sum = fmaf((float)r[ks].v[e], (float)r[ks].v[e], sum);
    return sqrtf(sum + other_half(sum));
}

template <typename T>
__device__ inline Pack<T> group_of(const f32x16 &s, int group) {
    Pack<T> p;
#pragma unroll
    for (int e = 0; e < kPack<T>; ++e) p.v[e] = (T)s[group * kPack<T> + e];
    return p;
}

// The floats of a block's 32 rows as the registers of multiply() stand for them.
__device__ inline f32x16 register_floats(LdsByte *floats, int block) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const int half = (threadIdx.x & (kWave - 1)) >> 5;
    f32x16 r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const auto v = lds_load<f32x4>(floats + half * 16 + (block * 32 + 8 * q) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[q * 4 + e] = v[e];
    }
    return r;
}

// A wave's lanes copy from[at] into LDS in their order, zeros where !in.
__device__ inline void copy_floats(LdsByte *lds, const float *from, int at, bool in) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)uniform((int64_t)from), 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)lds, 4,
                                             in ? (uint32_t)at * 4u : 0x80000000u, 0, 0, 0);
}

// The lane's row of D elements (times f) from the blocks of multiply().
template <bool WHOLE, typename OUT, int BLOCKS>
__device__ inline void store_row(OUT *row, const f32x16 (&acc)[BLOCKS], float f, int D) {
    const int half = (threadIdx.x & (kWave - 1)) >> 5;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = b * 32 + q * 8 + half * 4;
            OUT v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (OUT)(acc[b][q * 4 + e] * f);
            if (WHOLE ? d < D : d + 4 <= D) {
                __builtin_memcpy(row + d, v, sizeof(v));
            } else if constexpr (!WHOLE) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < D) row[d + e] = v[e];
            }
        }
}

// What the rounding of out leaves off, for the backward pass: dout.out is subtracted
// from every dout.v, where out's own rounding would weigh as much as ds's.
template <bool WHOLE, typename T, int BLOCKS>
__device__ inline void store_rest(T *row, f32x16 (&acc)[BLOCKS], float f, int D) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] = acc[b][i] * f - (float)(T)(acc[b][i] * f);
    store_row<WHOLE>(row, acc, 1.0f, D);
}

// What takes the powers of two out of the sums of ds again.
template <typename T>
__device__ inline float held_scale(float scale, float by) {
    return kHolds<T> ? scale * (0x1p-12f / by) : scale;
}

// What both query-side kernels know of a tile of packed rows.
template <typename T>
struct Queries {
    int m, packed;      // the lane's packed row, and how many there are
    int64_t row;        // its row, and head of the group
    int head;
    int seen;           // keys that it sees
    int seen_least, seen_most;      // over the wave's rows
    int64_t key0;       // the segment's first key
    int keys;

    __device__ inline void locate(const AttentionArgs &a, const Slot &s, int hk, int m0, int rows_ahead) {
        const Runs keyruns(a.key_offsets, a.S, a.K, 1);
        packed = s.packed;
        const int bound = keyruns.bound(s.run + (threadIdx.x & 1)), first = __builtin_amdgcn_readlane(bound, 0);
        key0 = first;
        keys = max(0, __builtin_amdgcn_readlane(bound, 1) - first);
        m = m0 + rows_ahead + (threadIdx.x & 31);
        const int mc = min(m, packed - 1), i = quotient(a.G, mc);
        row = (int64_t)s.row0 + i;
        head = hk * a.G.d + mc - i * a.G.d;
        const int ahead = keys - s.rows + 1;
        seen = sees(a, i, ahead);
        seen_least = uniform(sees(a, quotient(a.G, min(m0 + rows_ahead, packed - 1)), ahead));
        seen_most = uniform(sees(a, quotient(a.G, min(m0 + rows_ahead + 31, packed - 1)), ahead));
    }

    __device__ inline int sees(const AttentionArgs &a, int i, int ahead) const {
        return a.causal ? max(0, min(keys, i + ahead)) : keys;
    }

    __device__ inline bool exists() const { return m < packed; }
};

template <int LEN>
__device__ inline int seen_by_tile(const AttentionArgs &a, const Slot &s, int keys) {
    const int last = quotient(a.G, min((s.tile + 1) * LEN, s.packed) - 1);
    return a.causal ? max(0, min(keys, last + keys - s.rows + 1)) : keys;
}

// The lane's row of an operand, as the packs that the matrix steps take.
template <typename T, int DP>
using RowPacks = Pack<T>[Tile<T, DP>::kSteps];

// WHOLE: D is a multiple of a pack.
template <typename T, int DP, bool WHOLE>
__device__ inline void load_row(RowPacks<T, DP> &r, const T *row, int D, bool exists) {
    const int half = (threadIdx.x & (kWave - 1)) >> 5;
#pragma unroll
    for (int ks = 0; ks < Tile<T, DP>::kSteps; ++ks) {
        const int e = (2 * ks + half) * kPack<T>;
        if constexpr (WHOLE) {
            r[ks] = Pack<T>{};
            if (exists && e < D) r[ks] = load_pack(row + e);
        } else {
            r[ks] = load_pack(row + (exists && e < D ? e : 0), exists ? D - e : 0);
        }
    }
}

template <typename T, int WAVES>
constexpr int kTileRows = WAVES == 1 || sizeof(T) == 4 ? 32 : 64;

// Two waves to a SIMD where 256 registers hold one's rows, sums and, without
// direct copies, the tile on its way.
template <typename T, int DP, bool DIRECT>
constexpr int kQuerySide = sizeof(T) * DP > (DIRECT ? 256 : 128) ? 1 : 2;
template <typename T, int DP, bool DIRECT>
constexpr int kKeySide = sizeof(T) * DP > (DIRECT ? 128 : 64) ? 1 : 2;

// One wave's short segments are one tile: with one stage of it twice as many waves
// share a compute unit (4,096 graphs of 24 rows, 4 heads of 32 fp32, with gradients:
// 373 -> 309 us).  Forward, one row against long segments keeps two (32 rows, 100,003
// keys, 8 key heads of 128 bf16: 101 against 106 us).
template <int WAVES>
constexpr int kStagesOf = WAVES == 1 ? 1 : 2;

// Stages of two tiles each, arrays of their own (see Stages).
#define TILE_PAIRS(x, y, bytes, stages)                                             \
    __shared__ __attribute__((aligned(1024))) char x##0[bytes];                    \
    __shared__ __attribute__((aligned(1024))) char y##0[bytes];                    \
    __shared__ __attribute__((aligned(1024))) char x##1[stages == 1 ? 16 : bytes]; \
    __shared__ __attribute__((aligned(1024))) char y##1[stages == 1 ? 16 : bytes]; \
    LdsByte *const x[2] = {(LdsByte *)x##0, (LdsByte *)x##1};                      \
    LdsByte *const y[2] = {(LdsByte *)y##0, (LdsByte *)y##1}

// Walks the tiles [t0, t1) of two arrays: while tile t is used, tile t + 1 is
// on its way into the other stage (or, with one, into registers if !DIRECT).
template <bool DIRECT, int STAGES, typename LoadAll, typename PutAll, typename Use>
__device__ inline void walk(int t0, int t1, LoadAll load, PutAll put, Use use) {
    if (t0 >= t1) return;
    if constexpr (DIRECT && STAGES == 1) {
        for (int t = t0; t < t1; ++t) {
            load(t, 0);
            wait_copies<0>();
            use(t, 0);
            wait_copies<0>();
        }
    } else if constexpr (DIRECT) {
        load(t0, 0);
        auto step = [&](int t, int u) {
            wait_copies<0>();
            load(t + 1, 1 - u);                          // behind the last tile: zeros, or a tile that is not used
            use(t, u);
        };
        int t = t0;
        for (; t + 1 < t1; t += 2) {
            step(t, 0);
            step(t + 1, 1);
        }
        if (t < t1) step(t, 0);
        wait_copies<0>();
    } else if constexpr (STAGES == 1) {
        load(t0, 0);
        for (int t = t0; t < t1; ++t) {
            put(0);
            __syncthreads();
            if (t + 1 < t1) load(t + 1, 0);
            use(t, 0);
            __syncthreads();
        }
    } else {
        load(t0, 0);
        put(0);
        for (int t = t0; t < t1; t += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (t + u < t1) {
                    __syncthreads();
                    const bool more = t + u + 1 < t1;
                    if (more) load(t + u + 1, 1 - u);
                    use(t + u, u);
                    if (more) put(1 - u);
                }
        }
        __syncthreads();
    }
}

// ---- forward ----

template <typename T, int DP, int WAVES, bool DIRECT, int STAGES>
__global__ __launch_bounds__(WAVES * kWave, (kQuerySide<T, DP, DIRECT>)) void attention_kernel(AttentionArgs a,
                                                                                              unsigned total) {
    using L = Tile<T, DP>;
    constexpr int BM = 32 * WAVES, BN = kTileRows<T, WAVES>, NB = BN / 32;
    TILE_PAIRS(ktile, vtile, BN * L::kPitch, STAGES);
    const int wave = uniform((int)threadIdx.x / kWave), half = (threadIdx.x & (kWave - 1)) >> 5;
    const int D = (int)a.D;
    const RowReader<T, DP> rows;
    const TurnedReader<T, DP> turned;
    const Runs runs(a.offsets, a.S, a.R, a.G.d);
    const float c = a.scale * kLog2e;
    for (unsigned id = blockIdx.x; id < total; id += gridDim.x) {
        const unsigned heads = (unsigned)a.Hk, rest = id / heads, parts = (unsigned)a.parts;
        const int hk = (int)(id - rest * heads), part = (int)(rest % parts);
        Slot s = find<BM>(runs, (int)(rest / parts));
        if (s.tile >= s.tiles) continue;
        s.tile = s.tiles - 1 - s.tile;                   // causal: the longest first
        Queries<T> q;
        q.locate(a, s, hk, s.tile * BM, wave * 32);
        f32x16 acc[L::kBlocks] = {};
        float top = -INFINITY, sum = 0.0f;               // (top: less what weights are held times)
        if (s.run > 0 && s.run <= a.S) {
            const int tiles = (seen_by_tile<BM>(a, s, q.keys) + BN - 1) / BN;
            const int per = (tiles + a.parts - 1) / a.parts;
            const int t0 = part * per, t1 = min(tiles, t0 + per);
            RowPacks<T, DP> mine;
            load_row<T, DP, DIRECT>(mine, (const T *)a.q + q.row * a.ldq + q.head * D, D, q.exists());
            const T *k = (const T *)a.k + q.key0 * a.ldk + hk * D, *v = (const T *)a.v + q.key0 * a.ldv + hk * D;
            Fill<T, DP, BN, WAVES, DIRECT> fk, fv;
            fk.aim(KeyRows<T>{k, a.ldk, BN}, D, wave);
            fv.aim(KeyRows<T>{v, a.ldv, BN}, D, wave);
            __syncthreads();
            walk<DIRECT, STAGES>(
                t0, t1,
                [&](int t, int u) {
                    const int j = t * BN, left = q.keys - j;
                    fk.load(ktile[u], KeyRows<T>{k + j * a.ldk, a.ldk, left}, D, wave);
                    fv.load(vtile[u], KeyRows<T>{v + j * a.ldv, a.ldv, left}, D, wave);
                },
                [&](int u) {
                    fk.put(ktile[u], wave);
                    fv.put(vtile[u], wave);
                },
                [&](int t, int u) {
                    const int j0 = t * BN;
                    if (j0 >= q.seen_most) return;
                    f32x16 sc[NB] = {};
#pragma unroll
                    for (int ks = 0; ks < L::kSteps; ++ks)
#pragma unroll
                        for (int b = 0; b < NB; ++b) multiply<T>(mine[ks], rows.read(ktile[u], b, ks), sc[b]);
                    if constexpr (sizeof(T) == 2) {      // four reads ahead of the products
                        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
                        for (int i = 0; i < L::kSteps * NB; ++i) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        }
                    }
                    if (j0 + BN > q.seen_least) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (j0 + b * 32 + register_row(i) >= q.seen) sc[b][i] = -INFINITY;
                    }
                    float most = sc[0][0];
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) most = fmaxf(most, sc[b][i]);
                    most = fmaxf(most, other_half(most)) * c - kHeldBits<T>;
                    // The sums keep the maximum they were taken against until it
                    // grows by 2^8 (fp16: 2^3): weights up to 256 (8, held times 2^12)
                    // lose nothing, and most tiles rescale nothing.
                    if (__any(most > top + kGrowth<T>)) {
                        const float next = fmaxf(top, most);
                        const float f = next == -INFINITY ? 1.0f : exp2_of(top - next);
                        top = next;
                        sum *= f;
#pragma unroll
                        for (int b = 0; b < L::kBlocks; ++b) acc[b] *= f;
                    }
                    const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            sc[b][i] = exp2_of(fmaf(sc[b][i], c, -from));
                            sum += sc[b][i];
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int g = 0; g < L::kGroups; ++g) {
                            const Pack<T> p = group_of<T>(sc[b], g);
#pragma unroll
                            for (int d = 0; d < L::kBlocks; ++d)
                                multiply<T>(p, turned.read(vtile[u], b, g, d), acc[d]);
                        }
                });
        }
        sum += other_half(sum);
        const int64_t at = q.row * a.H + q.head, all = a.R * a.H;
        if (q.exists() && a.parts > 1) {
            store_row<DIRECT>(a.partial + (part * all + at) * D, acc, 1.0f, D);
            if (half == 0) {
                a.partial_top[part * all + at] = top;
                a.partial_sum[part * all + at] = sum;
            }
        } else if (q.exists()) {
            const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
            store_row<DIRECT>((T *)a.out + at * D, acc, f, D);
            if (a.rest) store_rest<DIRECT>((T *)a.rest + at * D, acc, f, D);
            if (a.lse && half == 0) a.lse[at] = sum == 0.0f ? INFINITY : top + log2f(sum);
        }
    }
}

// Joins the parts of the rows, four elements of one to a lane.
constexpr int kJoinThreads = 256;

template <typename T>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttentionArgs a) {
    const int D = (int)a.D, quads = (D + 3) / 4;
    const int64_t all = a.R * a.H;
    for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < all * quads;
         i += (int64_t)gridDim.x * kJoinThreads) {
        const int64_t at = i / quads;
        const int d = (int)(i - at * quads) * 4;
        // a part that sees nothing has the maximum -infinity and zeros
        float top = -INFINITY, sum = 0.0f, r[4] = {};
#pragma unroll 8
        for (int p = 0; p < a.parts; ++p) top = fmaxf(top, a.partial_top[p * all + at]);
        const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll 8
        for (int p = 0; p < a.parts; ++p) {
            const float weight = exp2_of(a.partial_top[p * all + at] - from);
            const Pack<float> v = load_pack(a.partial + (p * all + at) * D + d, D - d);
            sum = fmaf(a.partial_sum[p * all + at], weight, sum);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = fmaf(v.v[e], weight, r[e]);
        }
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < D) {
                const T v = (T)(r[e] * f);
                ((T *)a.out)[at * D + d + e] = v;
                if (a.rest) ((T *)a.rest)[at * D + d + e] = (T)(r[e] * f - (float)v);
            }
        if (a.lse && d == 0) a.lse[at] = sum == 0.0f ? INFINITY : top + log2f(sum);
    }
}

// ---- backward ----

// dq, and delta = dout.out of every row, which dk and dv take from here.
template <typename T, int DP, int WAVES, bool DIRECT>
__global__ __launch_bounds__(WAVES * kWave, (kQuerySide<T, DP, DIRECT>)) void attention_dq_kernel(AttentionArgs a,
                                                                                                 unsigned total) {
    using L = Tile<T, DP>;
    constexpr int BM = 32 * WAVES, BN = kTileRows<T, WAVES>, NB = BN / 32;
    TILE_PAIRS(ktile, vtile, BN * L::kPitch, kStagesOf<WAVES>);
    const int wave = uniform((int)threadIdx.x / kWave), half = (threadIdx.x & (kWave - 1)) >> 5;
    const int D = (int)a.D;
    const RowReader<T, DP> rows;
    const TurnedReader<T, DP> turned;
    const Runs runs(a.offsets, a.S, a.R, a.G.d);
    const float c = a.scale * kLog2e;
    for (unsigned id = blockIdx.x; id < total; id += gridDim.x) {
        const unsigned heads = (unsigned)a.Hk, rest = id / heads;
        const int hk = (int)(id - rest * heads);
        Slot s = find<BM>(runs, (int)rest);
        if (s.tile >= s.tiles) continue;
        s.tile = s.tiles - 1 - s.tile;
        Queries<T> q;
        q.locate(a, s, hk, s.tile * BM, wave * 32);
        const int64_t at = q.row * a.H + q.head;
        f32x16 acc[L::kBlocks] = {};
        HeldGradients<T> held;
        if (s.run > 0 && s.run <= a.S) {
            RowPacks<T, DP> mine, dout;
            load_row<T, DP, DIRECT>(dout, (const T *)a.dout + at * D, D, q.exists());
            float delta = 0.0f;
            for (const void *part : {(const void *)a.out, (const void *)a.rest}) {
                if (!part) break;
                load_row<T, DP, DIRECT>(mine, (const T *)part + at * D, D, q.exists());
#pragma unroll
                for (int ks = 0; ks < L::kSteps; ++ks)
#pragma unroll
                    for (int e = 0; e < kPack<T>; ++e) delta = fmaf((float)dout[ks].v[e], (float)mine[ks].v[e], delta);
            }
            delta += other_half(delta);
            const float lse = q.exists() ? a.lse[at] - kHeldBits<T> : INFINITY;
            if (q.exists() && half == 0) a.delta[at] = delta;
            if constexpr (kHolds<T>) {
                // what dk's kernel bounds its ds by; a row that is not finite bounds nothing
                const float length = length_of(dout), size = fabsf(delta);
                const float longest = wave_most(q.exists() && length < INFINITY ? length : 0.0f);
                const float largest = wave_most(q.exists() && size < INFINITY ? size : 0.0f);
                if ((threadIdx.x & (kWave - 1)) == 0) {
                    float *to = a.sizes + 2 * ((int64_t)id * WAVES + wave);
                    to[0] = longest;
                    to[1] = largest;
                }
                if (q.exists() && half == 0) a.held_lse[at] = lse;
            }
            if (a.dq) {
                load_row<T, DP, DIRECT>(mine, (const T *)a.q + q.row * a.ldq + q.head * D, D, q.exists());
                const int tiles = (seen_by_tile<BM>(a, s, q.keys) + BN - 1) / BN;
                const T *k = (const T *)a.k + q.key0 * a.ldk + hk * D, *v = (const T *)a.v + q.key0 * a.ldv + hk * D;
                Fill<T, DP, BN, WAVES, DIRECT> fk, fv;
                fk.aim(KeyRows<T>{k, a.ldk, BN}, D, wave);
                fv.aim(KeyRows<T>{v, a.ldv, BN}, D, wave);
                __syncthreads();
                walk<DIRECT, kStagesOf<WAVES>>(
                    0, tiles,
                    [&](int t, int u) {
                        const int j = t * BN, left = q.keys - j;
                        fk.load(ktile[u], KeyRows<T>{k + j * a.ldk, a.ldk, left}, D, wave);
                        fv.load(vtile[u], KeyRows<T>{v + j * a.ldv, a.ldv, left}, D, wave);
                    },
                    [&](int u) {
                        fk.put(ktile[u], wave);
                        fv.put(vtile[u], wave);
                    },
                    [&](int t, int u) {
                        const int j0 = t * BN;
                        if (j0 >= q.seen_most) return;
                        const bool border = j0 + BN > q.seen_least;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            f32x16 sc = {}, dp = {};
#pragma unroll
                            for (int ks = 0; ks < L::kSteps; ++ks) {
                                multiply<T>(mine[ks], rows.read(ktile[u], b, ks), sc);
                                multiply<T>(dout[ks], rows.read(vtile[u], b, ks), dp);
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) sc[i] = exp2_of(fmaf(sc[i], c, -lse));
                            if (border) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (j0 + b * 32 + register_row(i) >= q.seen) sc[i] = 0.0f;
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                sc[i] *= kHolds<T> ? fmaf(dp[i], held.by, -delta * held.by) : dp[i] - delta;
                            held.follow(sc, acc);
#pragma unroll
                            for (int g = 0; g < L::kGroups; ++g) {
                                const Pack<T> ds = group_of<T>(sc, g);
#pragma unroll
                                for (int d = 0; d < L::kBlocks; ++d)
                                    multiply<T>(ds, turned.read(ktile[u], b, g, d), acc[d]);
                            }
                        }
                    });
            }
        } else if (q.exists() && half == 0) {
            a.delta[at] = 0.0f;
        }
        if (a.dq && q.exists())
            store_row<DIRECT>((T *)a.dq + at * D, acc, held_scale<T>(a.scale, held.by), D);
    }
}

// Parts that the packed rows of a key tile are taken in: they differ in how many
// see the tile, and a part is to be a third of a compute unit's share of the call.
__device__ inline int parts_of_tile(const AttentionArgs &a, int tiles, int tile_rows) {
    return max(1, min(a.key_parts, (int)(((int64_t)tiles * tile_rows + a.part_rows - 1) / a.part_rows)));
}

// What a key tile knows of the rows of its segment.
struct SeenBy {
    int64_t row0;
    int packed, start, tiles;     // tiles of packed rows from `start` on see the tile
    int64_t behind;

    __device__ inline SeenBy(const AttentionArgs &a, const Slot &s, int key, int tile_rows) {
        const Runs queries(a.offsets, a.S, a.R, 1);
        const int bound = queries.bound(s.run + (threadIdx.x & 1)), from = __builtin_amdgcn_readlane(bound, 0);
        row0 = from;
        const int rows = max(0, __builtin_amdgcn_readlane(bound, 1) - from);
        packed = rows * a.G.d;
        behind = a.causal ? (int64_t)rows - s.rows : INT32_MIN;
        start = first(a, key) / tile_rows;
        tiles = max(0, (packed + tile_rows - 1) / tile_rows - start);
    }

    // Packed rows from this one on see key j of the segment.
    __device__ inline int first(const AttentionArgs &a, int j) const {
        return (int)max(int64_t(0), min((int64_t)packed, (j + behind) * a.G.d));
    }
};

// What dk and dv read of a tile of packed rows: q and dout in LDS, and the rows'
// lse and delta.
template <typename T, int DP, int BN, int WAVES, bool DIRECT>
struct RowTiles {
    const AttentionArgs &a;
    int64_t row0;
    int hk, packed, wave;
    Fill<T, DP, BN, WAVES, DIRECT> fq, fd;
    float lse, delta;

    __device__ inline RowTiles(const AttentionArgs &args, int64_t first, int head, int rows, int w)
        : a(args), row0(first), hk(head), packed(rows), wave(w), lse(0.0f), delta(0.0f) {
        aim(0);
    }

    __device__ inline PackedRows<T> q(int m0) const {
        const int i0 = quotient(a.G, m0);
        return {(const T *)a.q + (row0 + i0) * a.ldq + hk * a.G.d * a.D, a.ldq, packed - m0, m0, i0, (int)a.D, a.G};
    }
    __device__ inline PackedRows<T> dout(int m0) const {
        const int i0 = quotient(a.G, m0);
        return {(const T *)a.dout + ((row0 + i0) * a.H + hk * a.G.d) * a.D, a.H * a.D, packed - m0, m0, i0, (int)a.D,
                a.G};
    }

    __device__ inline void aim(int m0) {
        fq.aim(q(m0), (int)a.D, wave);
        fd.aim(dout(m0), (int)a.D, wave);
    }

    __device__ inline void load(int t, LdsByte *qt, LdsByte *dt, LdsByte *lse_of, LdsByte *delta_of) {
        const int m0 = t * BN, left = packed - m0;
        // tiles of whole groups stand alike, one ld apart
        if (DIRECT && BN % a.G.d) aim(m0);
        fq.load(qt, q(m0), (int)a.D, wave);
        fd.load(dt, dout(m0), (int)a.D, wave);
        // one lane to a row; rows that do not exist take zeros, and their
        // operands are zeros
        if (wave == 0) {
            const int i0 = quotient(a.G, m0), m = m0 + (int)threadIdx.x, i = quotient(a.G, m);
            const bool in = (int)threadIdx.x < min(BN, left);
            const int64_t from = (row0 + i0) * a.H + hk * a.G.d;
            const int at = (int)((i - i0) * a.H) + m - i * a.G.d;
            if constexpr (DIRECT) {
                copy_floats(lse_of, (kHolds<T> ? a.held_lse : a.lse) + from, at, in);
                copy_floats(delta_of, a.delta + from, at, in);
            } else {
                lse = in ? (kHolds<T> ? a.held_lse : a.lse)[from + at] : 0.0f;
                delta = in ? a.delta[from + at] : 0.0f;
            }
        }
    }

    __device__ inline void put(LdsByte *qt, LdsByte *dt, LdsByte *lse_of, LdsByte *delta_of) {
        fq.put(qt, wave);
        fd.put(dt, wave);
        if (!DIRECT && wave == 0) {
            ((__attribute__((address_space(3))) float *)lse_of)[threadIdx.x] = lse;
            ((__attribute__((address_space(3))) float *)delta_of)[threadIdx.x] = delta;
        }
    }
};

// The sums of a wave's 32 keys over 32-row blocks of packed rows.
template <typename T, int DP>
struct KeySums {
    using L = Tile<T, DP>;
    struct TurnedRows {
        Pack<T> at[L::kGroups][L::kBlocks];
    };
    struct Weights {
        Pack<T> p[L::kGroups], ds[L::kGroups];
    };
    f32x16 dk[L::kBlocks] = {}, dv[L::kBlocks] = {};
    RowPacks<T, DP> k, v;
    RowReader<T, DP> rows;
    TurnedReader<T, DP> turned;
    float c;
    float by = 1.0f;

    // ds of the lane's key is held times a power of two `by` in fp16: |ds| <= |dout| |v| +
    // |dout.out| over the rows of the segment is brought to 2^15 at most (2^12 p among it).
    // By a bound and not by the largest so far, whose branch parts the products from the
    // reads ahead of them (8,192 causal rows, 16 heads of 128 over 4: 448 us, 368 with the
    // bound, 341 with ds as it is).  ds of 2^-29 of the bound keep eleven bits: of even
    // weights over 32,768 keys, rows with a thousandth of the longest dout.
    __device__ inline void hold(const AttentionArgs &a, int run, int hk, int64_t row0, int packed) {
        if constexpr (kHolds<T>) {
            // dq's waves of the segment's rows: those of its tiles, slot by slot
            const int waves = a.query_rows / 32, tiles = (packed + a.query_rows - 1) / a.query_rows;
            const int64_t slot = row0 * a.G.d / a.query_rows + run;
            float longest = 0.0f, largest = 0.0f;
            for (int i = threadIdx.x & (kWave - 1); i < tiles * waves; i += kWave) {
                const float *at = a.sizes + 2 * (((slot + i / waves) * a.Hk + hk) * waves + i % waves);
                longest = fmaxf(longest, at[0]);
                largest = fmaxf(largest, at[1]);
            }
            const float most = wave_most(longest) * length_of(v) + wave_most(largest);
            if (most > 0.0f && most < INFINITY) by = ldexpf(1.0f, 3 - __builtin_amdgcn_frexp_expf(most));
        }
    }

    __device__ inline void read(RowPacks<T, DP> &r, LdsByte *tile, int b) const {
#pragma unroll
        for (int ks = 0; ks < L::kSteps; ++ks) r[ks] = rows.read(tile, b, ks);
    }
    __device__ inline void read(TurnedRows &r, LdsByte *tile, int b) const {
#pragma unroll
        for (int g = 0; g < L::kGroups; ++g)
#pragma unroll
            for (int e = 0; e < L::kBlocks; ++e) r.at[g][e] = turned.read(tile, b, g, e);
    }
    static __device__ inline void product(const RowPacks<T, DP> &mine, const RowPacks<T, DP> &r, f32x16 &to) {
        to = f32x16{};
#pragma unroll
        for (int ks = 0; ks < L::kSteps; ++ks) multiply<T>(mine[ks], r[ks], to);
    }
    // Rows ahead of `from` of a block that starts at m0 do not see the lane's key.
    static __device__ inline void hide(f32x16 &sc, int m0, int from) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (m0 + register_row(i) < from) sc[i] = -INFINITY;
    }
    __device__ inline void probabilities(f32x16 &sc, LdsByte *lse_of, int b) const {
        const f32x16 lse = register_floats(lse_of, b);
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[i] = exp2_of(fmaf(sc[i], c, -lse[i]));
    }
    // ds from the probabilities and dp
    __device__ inline void gradients(f32x16 &dp, const f32x16 &sc, const f32x16 &delta) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) dp[i] = sc[i] * (dp[i] - delta[i]);
        if constexpr (kHolds<T>) dp *= by;
    }
    static __device__ inline void add(f32x16 (&to)[L::kBlocks], const Pack<T> (&w)[L::kGroups], const TurnedRows &r) {
#pragma unroll
        for (int g = 0; g < L::kGroups; ++g)
#pragma unroll
            for (int e = 0; e < L::kBlocks; ++e) multiply<T>(w[g], r.at[g][e], to[e]);
    }

    // A block whose rows of q have been read: each product runs beside the reads
    // of the next one's operand and the arithmetic that does not wait for it.
    // ahead() reads q of the block after it; border: see hide().
    template <typename Ahead>
    __device__ inline void block(RowPacks<T, DP> &q, LdsByte *qt, LdsByte *dt, LdsByte *lse_of, LdsByte *delta_of,
                                 int b, bool border, int m0, int from, Ahead ahead) {
        RowPacks<T, DP> d;
        TurnedRows dturned, qturned;
        f32x16 sc, dp;
        Weights w;
        read(d, dt, b);
        product(k, q, sc);
        if (border) hide(sc, m0, from);
        __builtin_amdgcn_sched_barrier(0);
        read(dturned, dt, b);
        product(v, d, dp);
        probabilities(sc, lse_of, b);
#pragma unroll
        for (int g = 0; g < L::kGroups; ++g) w.p[g] = group_of<T>(sc, g);
        spread();
        __builtin_amdgcn_sched_barrier(0);
        read(qturned, qt, b);
        add(dv, w.p, dturned);
        gradients(dp, sc, register_floats(delta_of, b));
#pragma unroll
        for (int g = 0; g < L::kGroups; ++g) w.ds[g] = group_of<T>(dp, g);
        spread();
        __builtin_amdgcn_sched_barrier(0);
        ahead();
        add(dk, w.ds, qturned);
        __builtin_amdgcn_sched_barrier(0);
    }

    // Reads first, then the products with the rest spread between them.
    static __device__ inline void spread() {
        constexpr int kProducts = L::kSteps;
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int i = 0; i < kProducts; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
        }
    }
};

// dk and dv: the block's keys against the packed rows that see them.
//
// Where one wave to a SIMD holds its keys and their sums (16-bit rows of more than
// 64 elements), it reads ahead: a block's turned rows while its exponentials run,
// and the next block's rows while the products with the turned ones run.
template <typename T, int DP, int WAVES, bool DIRECT>
__global__ __launch_bounds__(WAVES * kWave, (kKeySide<T, DP, DIRECT>)) void attention_dkdv_kernel(AttentionArgs a,
                                                                                                 unsigned total) {
    using L = Tile<T, DP>;
    using K = KeySums<T, DP>;
    constexpr int BM = 32 * WAVES, BN = kTileRows<T, WAVES>, NB = BN / 32;
    constexpr bool kAhead = DIRECT && sizeof(T) == 2 && WAVES == 4 && DP > 64;
    TILE_PAIRS(qtile, dtile, BN * L::kPitch, kStagesOf<WAVES>);
    TILE_PAIRS(lse_of, delta_of, kWave * 4, kStagesOf<WAVES>);
    const int wave = uniform((int)threadIdx.x / kWave);
    const int D = (int)a.D;
    const Runs runs(a.key_offsets, a.S, a.K, 1);
    for (unsigned id = blockIdx.x; id < total; id += gridDim.x) {
        const unsigned heads = (unsigned)a.Hk, rest = id / heads, most = (unsigned)a.key_parts;
        // tiles use few of their parts: they start at another one in each, so that
        // the XCDs, which take blocks in turn, get alike
        const int hk = (int)(id - rest * heads), slot = (int)(rest / most), part = (int)((rest + slot) % most);
        const Slot s = find<BM>(runs, slot);
        if (s.tile >= s.tiles) continue;
        const int j0 = s.tile * BM + wave * 32, j = j0 + (threadIdx.x & 31);
        const bool exists = j < s.rows, inside = s.run > 0 && s.run <= a.S;
        const SeenBy by(a, s, s.tile * BM, BN);
        const int parts = inside ? parts_of_tile(a, by.tiles, BN) : 1;
        if (part >= parts) continue;
        K sums;
        sums.c = a.scale * kLog2e;
        if (inside) {
            const int mine_from = by.first(a, j), wave_from = by.first(a, j0), wave_full = by.first(a, j0 + 31);
            const int per = (by.tiles + parts - 1) / parts;
            const int t0 = by.start + min(by.tiles, part * per), t1 = min(by.start + by.tiles, t0 + per);
            const int64_t key = (int64_t)s.row0 + min(j, s.rows - 1);
            load_row<T, DP, DIRECT>(sums.k, (const T *)a.k + key * a.ldk + hk * D, D, exists);
            load_row<T, DP, DIRECT>(sums.v, (const T *)a.v + key * a.ldv + hk * D, D, exists);
            sums.hold(a, s.run, hk, by.row0, by.packed);
            RowTiles<T, DP, BN, WAVES, DIRECT> tiles(a, by.row0, hk, by.packed, wave);
            __syncthreads();
            if constexpr (kAhead) {
                auto load = [&](int t, int u) { tiles.load(t, qtile[u], dtile[u], lse_of[u], delta_of[u]); };
                RowPacks<T, DP> q;
                if (t0 < t1) {
                    load(t0, 0);
                    wait_copies<0>();
                    load(t0 + 1, 1);
                    sums.read(q, qtile[0], 0);
                    auto tile = [&](int t, int u) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int m0 = t * BN + b * 32;
                            sums.block(q, qtile[u], dtile[u], lse_of[u], delta_of[u], b, m0 < wave_full, m0, mine_from,
                                       [&] {
                                           if (b == NB - 1) {
                                               // this tile is read out, and the next one here
                                               wait_copies<0>();
                                               load(t + 2, u);
                                               sums.read(q, qtile[1 - u], 0);
                                           } else {
                                               sums.read(q, qtile[u], b + 1);
                                           }
                                       });
                        }
                    };
                    int t = t0;
                    for (; t + 1 < t1; t += 2) {
                        tile(t, 0);
                        tile(t + 1, 1);
                    }
                    if (t < t1) tile(t, 0);
                    wait_copies<0>();
                }
            } else {
                walk<DIRECT, kStagesOf<WAVES>>(
                    t0, t1, [&](int t, int u) { tiles.load(t, qtile[u], dtile[u], lse_of[u], delta_of[u]); },
                    [&](int u) { tiles.put(qtile[u], dtile[u], lse_of[u], delta_of[u]); },
                    [&](int t, int u) {
                        if (t * BN + BN <= wave_from) return;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int m0 = t * BN + b * 32;
                            f32x16 sc = {}, dp = {};
#pragma unroll
                            for (int ks = 0; ks < L::kSteps; ++ks) {
                                multiply<T>(sums.k[ks], sums.rows.read(qtile[u], b, ks), sc);
                                multiply<T>(sums.v[ks], sums.rows.read(dtile[u], b, ks), dp);
                            }
                            if (m0 < wave_full) K::hide(sc, m0, mine_from);
                            sums.probabilities(sc, lse_of[u], b);
                            sums.gradients(dp, sc, register_floats(delta_of[u], b));
#pragma unroll
                            for (int g = 0; g < L::kGroups; ++g) {
                                const Pack<T> p = group_of<T>(sc, g), ds = group_of<T>(dp, g);
#pragma unroll
                                for (int e = 0; e < L::kBlocks; ++e) {
                                    multiply<T>(p, sums.turned.read(dtile[u], b, g, e), sums.dv[e]);
                                    multiply<T>(ds, sums.turned.read(qtile[u], b, g, e), sums.dk[e]);
                                }
                            }
                        }
                    });
            }
        }
        const int64_t at = (((int64_t)s.row0 + j) * a.Hk + hk) * D, shift = part * a.K * a.Hk * a.D;
        const float fk = held_scale<T>(a.scale, sums.by), fv = kHolds<T> ? 0x1p-12f : 1.0f;
        if (exists && parts > 1) {
            if (a.dk) store_row<DIRECT>(a.partial_dk + shift + at, sums.dk, fk, D);
            if (a.dv) store_row<DIRECT>(a.partial_dv + shift + at, sums.dv, fv, D);
        } else if (exists) {
            if (a.dk) store_row<DIRECT>((T *)a.dk + at, sums.dk, fk, D);
            if (a.dv) store_row<DIRECT>((T *)a.dv + at, sums.dv, fv, D);
        }
    }
}

// Adds the parts of dk and dv in their order, a block to 16 keys of a tile and head.
constexpr int kAddThreads = 256, kAddKeys = 16;

template <typename T, int LEN, int ROWS>
__global__ __launch_bounds__(kAddThreads) void attention_add_kernel(AttentionArgs a, unsigned total) {
    const Runs runs(a.key_offsets, a.S, a.K, 1);
    const int D = (int)a.D, quads = (D + 3) / 4;
    const int64_t all = a.K * a.Hk * D;
    for (unsigned id = blockIdx.x; id < total; id += gridDim.x) {
        const unsigned heads = (unsigned)a.Hk, rest = id / heads, slot = rest / (LEN / kAddKeys);
        const int hk = (int)(id - rest * heads), first = (int)(rest - slot * (LEN / kAddKeys)) * kAddKeys;
        const Slot s = find<LEN>(runs, (int)slot);
        if (s.tile >= s.tiles || s.run == 0 || s.run > a.S) continue;
        const SeenBy by(a, s, s.tile * LEN, ROWS);
        const int parts = parts_of_tile(a, by.tiles, ROWS);
        if (parts == 1) continue;
        const int key = s.tile * LEN + first, keys = min(kAddKeys, s.rows - key);
        for (int i = threadIdx.x; i < 2 * keys * quads; i += kAddThreads) {
            const bool second = i >= keys * quads;
            T *to = (T *)(second ? a.dv : a.dk);
            if (!to) continue;
            const int in = second ? i - keys * quads : i, row = in / quads, d = (in - row * quads) * 4;
            const int64_t at = (((int64_t)s.row0 + key + row) * a.Hk + hk) * D + d;
            const float *from = (second ? a.partial_dv : a.partial_dk) + at;
            float sum[4] = {};
            for (int p = 0; p < parts; ++p, from += all) {
                const Pack<float> v = load_pack(from, D - d);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] += v.v[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D) to[at + e] = (T)sum[e];
        }
    }
}

// ---- the launches ----

constexpr int64_t kMaxBlocks = 1 << 20;

// Tiles of LEN rows: the most that the runs of a call can have.
inline unsigned slots(int64_t packed, int64_t S, int len) { return (unsigned)(packed / len + S + 2); }

template <typename T, int DP, int WAVES, bool DIRECT>
hipError_t forward_launch(const AttentionArgs &a, hipStream_t s) {
    const unsigned total = slots(a.R * a.G.d, a.S, 32 * WAVES) * (unsigned)(a.Hk * a.parts);
    const unsigned blocks = (unsigned)std::min<int64_t>(total, kMaxBlocks);
    if constexpr (WAVES == 1) {
        if (a.short_keys) {
            attention_kernel<T, DP, WAVES, DIRECT, 1><<<blocks, WAVES * kWave, 0, s>>>(a, total);
            return hipGetLastError();
        }
    }
    attention_kernel<T, DP, WAVES, DIRECT, 2><<<blocks, WAVES * kWave, 0, s>>>(a, total);
    return hipGetLastError();
}

template <typename T, int DP, int WAVES, bool DIRECT>
hipError_t dq_launch(const AttentionArgs &a, hipStream_t s) {
    const unsigned total = slots(a.R * a.G.d, a.S, 32 * WAVES) * (unsigned)a.Hk;
    const unsigned blocks = (unsigned)std::min<int64_t>(total, kMaxBlocks);
    attention_dq_kernel<T, DP, WAVES, DIRECT><<<blocks, WAVES * kWave, 0, s>>>(a, total);
    return hipGetLastError();
}

template <typename T, int DP, int WAVES, bool DIRECT>
hipError_t dkdv_launch(const AttentionArgs &a, hipStream_t s) {
    const unsigned total = slots(a.K, a.S, 32 * WAVES) * (unsigned)(a.Hk * a.key_parts);
    const unsigned blocks = (unsigned)std::min<int64_t>(total, kMaxBlocks);
    attention_dkdv_kernel<T, DP, WAVES, DIRECT><<<blocks, WAVES * kWave, 0, s>>>(a, total);
    return hipGetLastError();
}

template <typename T, int DP, int WAVES, bool DIRECT>
hipError_t launch_one(const AttentionArgs &a, AttentionPass pass, hipStream_t s) {
    if (pass == AttentionPass::kForward) return forward_launch<T, DP, WAVES, DIRECT>(a, s);
    if (pass == AttentionPass::kQueries) return dq_launch<T, DP, WAVES, DIRECT>(a, s);
    return dkdv_launch<T, DP, WAVES, DIRECT>(a, s);
}

template <typename T, int DP>
hipError_t launch_width(const AttentionArgs &a, AttentionPass pass, bool large, bool direct, hipStream_t s) {
    if (large) return direct ? launch_one<T, DP, 4, true>(a, pass, s) : launch_one<T, DP, 4, false>(a, pass, s);
    return direct ? launch_one<T, DP, 1, true>(a, pass, s) : launch_one<T, DP, 1, false>(a, pass, s);
}

}  // namespace

template <typename T>
hipError_t launch_attention_pass(const AttentionArgs &a, AttentionPass pass, bool large, bool direct, hipStream_t s) {
    if (a.D <= 32) return launch_width<T, 32>(a, pass, large, direct, s);
    if (a.D <= 64) return launch_width<T, 64>(a, pass, large, direct, s);
    if (a.D <= 96) return launch_width<T, 96>(a, pass, large, direct, s);
    return launch_width<T, 128>(a, pass, large, direct, s);
}

template <typename T>
hipError_t launch_attention_join(const AttentionArgs &a, hipStream_t s) {
    const int64_t blocks = (a.R * a.H * ((a.D + 3) / 4) + kJoinThreads - 1) / kJoinThreads;
    attention_join_kernel<T><<<(unsigned)std::min(blocks, kMaxBlocks), kJoinThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int WAVES>
hipError_t add_launch(const AttentionArgs &a, hipStream_t s) {
    const unsigned total = slots(a.K, a.S, 32 * WAVES) * (unsigned)a.Hk * (32 * WAVES / kAddKeys);
    const unsigned blocks = (unsigned)std::min<int64_t>(total, kMaxBlocks);
    attention_add_kernel<T, 32 * WAVES, kTileRows<T, WAVES>><<<blocks, kAddThreads, 0, s>>>(a, total);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_attention_add(const AttentionArgs &a, bool large, hipStream_t s) {
    return large ? add_launch<T, 4>(a, s) : add_launch<T, 1>(a, s);
}

#define ATTENTION_OF(T)                                                                                          \
    template hipError_t launch_attention_pass<T>(const AttentionArgs &, AttentionPass, bool, bool, hipStream_t); \
    template hipError_t launch_attention_join<T>(const AttentionArgs &, hipStream_t);                            \
    template hipError_t launch_attention_add<T>(const AttentionArgs &, bool, hipStream_t)

}  // namespace gspmm
