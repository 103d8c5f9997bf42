// The routed exchange: rows sorted by expert, copied into that order, and the
// experts' rows summed back with weights, with the gradients of both.
//
//  * Route.  The pairs p = t * k + j are sorted by expert, stably; pairs whose
//    expert is outside [0, E) come last.  A counting sort: a pair's place is
//    (pairs of smaller experts) + (pairs of its expert in earlier blocks and
//    waves) + (its rank inside its wave).  The rank comes from ballots: the
//    lanes of a wave that hold the same key are found with one ballot per key
//    bit, so equal keys keep their order and no atomic decides a place.
//  * Dispatch: row p of the output is x[order[p] / k].  The output is one
//    contiguous array, written in order in aligned 16-byte packs; the k copies
//    of a row of x are read at different times, mostly from the Infinity Cache.
//  * Combine: out[t] = sum_j weight[t, j] * rows[position[t, j]], j ascending,
//    one fused multiply-add per term.  With no weights it is dispatch's
//    gradient.
//  * Combine's gradients: drows[p] = weight[q] * dout[q / k] and dweight[q] =
//    <rows[p], dout[q / k]> for the pair q = order[p], one pass over both.
//
// All three move bytes and nothing else.  Calls that move more than half of
// the 256 MB Infinity Cache use non-temporal stores, and non-temporal loads
// for rows that are read once when rows are whole 16-byte groups (lanes of
// other rows share cache lines).  Measured: 16,384 x 2048 bf16 rows, k = 4:
// dispatch walked by source row 118 us, with non-temporal stores 92 us, by
// output row with them 77 us (4.3 TB/s of x once and the output); combine 77
// us with plain, 72 us with non-temporal stores, 69 us with loads as well (4.9
// TB/s); gradients by source row 134 us, by output row 118 us (5.1 TB/s).
// 50,021 x 1433 fp16 rows, k = 3: dispatch by source row 239 us, by output
// row in packs of one row 218 us, in aligned packs 190 us (at width 1432, with
// aligned loads, 143 us); combine 143, 136 and 147 us.  Those are figures of one
// occasion each.  Loops of one call as the kernels stand: dispatch 140, combine
// 132, gradients 205 us, at width 1432 125, 110 and 196 us; dispatch between
// other kernels 167 us.
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kWave = 64;

// ------------------------------------------------------------------ route

__device__ inline int route_key(int64_t e, int E) { return e >= 0 && e < E ? (int)e : E; }

// Exclusive sum of v over the block's threads; total in *total.
template <int THREADS>
__device__ inline int block_exclusive(int v, int *sh, int *total) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int incl = v;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int up = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += up;
    }
    if (lane == kWave - 1) sh[wave] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w) {
        if (w < wave) before += sh[w];
        all += sh[w];
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
}

// Keys of the wave's GROUPS x 64 consecutive pairs from `first`, and each
// pair's rank among the wave's pairs of the same key; count[key] ends as the
// wave's number of pairs of each key (zeroed by the caller).
template <int GROUPS>
__device__ inline void rank_in_wave(const RouteArgs &a, int64_t first, int bits, int *count, int (&key)[GROUPS],
                                    int (&rank)[GROUPS]) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint64_t below = (uint64_t(1) << lane) - 1;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        const int64_t p = first + g * kWave + lane;
        key[g] = p < a.pairs ? route_key(a.expert[p], a.E) : -1;
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        uint64_t same = __ballot(key[g] >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((key[g] >> b) & 1);
            same &= ((key[g] >> b) & 1) ? set : ~set;
        }
        int before = 0;
        if (key[g] >= 0) before = count[key[g]];
        rank[g] = before + __popcll(same & below);
        // the lanes' reads above come before the group's one write per key
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (key[g] >= 0 && (same & below) == 0) count[key[g]] = before + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int GROUPS>
__device__ inline void write_places(const RouteArgs &a, int64_t first, const int *base, const int (&key)[GROUPS],
                                    const int (&rank)[GROUPS]) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        const int64_t p = first + g * kWave + lane;
        if (key[g] < 0) continue;
        const int place = base[key[g]] + rank[g];
        a.position[p] = place;
        a.order[place] = (int)p;
    }
}

// The whole route in one block of 16 waves: small batches, where launches
// are what costs.
template <int GROUPS>
__global__ __launch_bounds__(1024) void route_one_kernel(RouteArgs a, int bits) {
    constexpr int kThreads = 1024, kWaves = kThreads / kWave;
    extern __shared__ int lds[];
    __shared__ int sh[kWaves];
    const int keys = a.E + 1, wave = threadIdx.x / kWave;
    int *count = lds + wave * keys;
    for (int i = threadIdx.x; i < kWaves * keys; i += kThreads) lds[i] = 0;
    __syncthreads();
    int key[GROUPS], rank[GROUPS];
    const int64_t first = (int64_t)wave * GROUPS * kWave;
    rank_in_wave<GROUPS>(a, first, bits, count, key, rank);
    __syncthreads();
    const int e = threadIdx.x;                       // keys <= 1024: one key per thread
    int mine = 0;
    if (e < keys)
        for (int w = 0; w < kWaves; ++w) mine += lds[w * keys + e];
    int total;
    int at = block_exclusive<kThreads>(mine, sh, &total);
    if (e < keys) {
        a.offsets[e] = at;
        for (int w = 0; w < kWaves; ++w) {
            const int c = lds[w * keys + e];
            lds[w * keys + e] = at;
            at += c;
        }
    }
    __syncthreads();
    write_places<GROUPS>(a, first, count, key, rank);
}

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kRouteGroups = 8;
constexpr int kRouteTile = kRouteThreads * kRouteGroups;   // pairs of one tile
constexpr int kRouteMaxBlocks = 1024;

// hist[key][block]: pairs of each key in the block's tiles.
__global__ __launch_bounds__(kRouteThreads) void route_count_kernel(RouteArgs a, int64_t tiles_per_block) {
    extern __shared__ int lds[];
    const int keys = a.E + 1;
    for (int i = threadIdx.x; i < keys; i += kRouteThreads) lds[i] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * tiles_per_block * kRouteTile;
    const int64_t p1 = min(a.pairs, p0 + tiles_per_block * kRouteTile);
    for (int64_t q0 = p0; q0 < p1; q0 += kRouteTile) {           // a tile's loads are in flight together
        int key[kRouteGroups];
#pragma unroll
        for (int g = 0; g < kRouteGroups; ++g) {
            const int64_t p = q0 + g * kRouteThreads + threadIdx.x;
            key[g] = p < p1 ? route_key(a.expert[p], a.E) : -1;
        }
#pragma unroll
        for (int g = 0; g < kRouteGroups; ++g)
            if (key[g] >= 0) atomicAdd(&lds[key[g]], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < keys; i += kRouteThreads)
        a.workspace[(int64_t)i * gridDim.x + blockIdx.x] = lds[i];
}

// Block `key`: exclusive sum of hist[key] over the blocks, in place, and its total.
__global__ __launch_bounds__(kRouteThreads) void route_scan_kernel(int *hist, int nblocks, int *total_of) {
    __shared__ int sh[kRouteWaves];
    int *row = hist + (int64_t)blockIdx.x * nblocks;
    int run = 0;
    for (int b0 = 0; b0 < nblocks; b0 += kRouteThreads) {
        const int b = b0 + threadIdx.x;
        const int v = b < nblocks ? row[b] : 0;
        int total;
        const int at = block_exclusive<kRouteThreads>(v, sh, &total);
        if (b < nblocks) row[b] = run + at;
        run += total;
    }
    if (threadIdx.x == 0) total_of[blockIdx.x] = run;
}

// SORTED: the pairs of a tile are sorted in LDS first, so that `order` is
// written in runs and not in 4-byte stores all over the array.
template <bool SORTED>
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a, const int *hist, const int *total_of,
                                                                    int bits, int64_t tiles_per_block) {
    extern __shared__ int lds[];             // base[keys], count[kRouteWaves][keys]; SORTED: shift[keys] and the
    __shared__ int sh[kRouteWaves];          // tile's place[kRouteTile] and pair[kRouteTile] in key order
    const int keys = a.E + 1, wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    int *base = lds, *counts = lds + keys, *shift = counts + kRouteWaves * keys, *place = shift + keys;
    uint16_t *pair = (uint16_t *)(place + kRouteTile);
    const int first = wave * kRouteGroups * kWave;
    // offsets: each thread takes a run of keys
    const int per = (keys + kRouteThreads - 1) / kRouteThreads;
    const int k0 = min(keys, (int)threadIdx.x * per), k1 = min(keys, k0 + per);
    int mine = 0;
    for (int i = k0; i < k1; ++i) mine += total_of[i];
    int total;
    int at = block_exclusive<kRouteThreads>(mine, sh, &total);
    for (int i = k0; i < k1; ++i) {
        if (blockIdx.x == 0) a.offsets[i] = at;
        base[i] = at + hist[(int64_t)i * gridDim.x + blockIdx.x];
        at += total_of[i];
    }
    for (int64_t t = 0; t < tiles_per_block; ++t) {
        const int64_t tile0 = ((int64_t)blockIdx.x * tiles_per_block + t) * kRouteTile;
        if (tile0 >= a.pairs) break;
        __syncthreads();
        for (int i = threadIdx.x; i < kRouteWaves * keys; i += kRouteThreads) counts[i] = 0;
        __syncthreads();
        int key[kRouteGroups], rank[kRouteGroups];
        rank_in_wave<kRouteGroups>(a, tile0 + first, bits, counts + wave * keys, key, rank);
        __syncthreads();
        if constexpr (SORTED) {
            // counts: each wave's first slot of a key; shift: from a slot to its place
            int inside = 0;
            for (int i = k0; i < k1; ++i)
                for (int w = 0; w < kRouteWaves; ++w) inside += counts[w * keys + i];
            int slot = block_exclusive<kRouteThreads>(inside, sh, &total);
            for (int i = k0; i < k1; ++i) {
                const int start = slot;
                for (int w = 0; w < kRouteWaves; ++w) {
                    const int c = counts[w * keys + i];
                    counts[w * keys + i] = slot;
                    slot += c;
                }
                shift[i] = base[i] - start;
                base[i] += slot - start;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kRouteGroups; ++g) {
                if (key[g] < 0) continue;
                const int q = first + g * kWave + lane, s = counts[wave * keys + key[g]] + rank[g];
                const int to = s + shift[key[g]];
                a.position[tile0 + q] = to;
                place[s] = to;
                pair[s] = (uint16_t)q;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kRouteGroups; ++g) {
                const int s = g * kRouteThreads + threadIdx.x;
                if (s < total) a.order[place[s]] = (int)(tile0 + pair[s]);
            }
        } else {
            for (int i = threadIdx.x; i < keys; i += kRouteThreads) {
                int run = base[i];
                for (int w = 0; w < kRouteWaves; ++w) {
                    const int c = counts[w * keys + i];
                    counts[w * keys + i] = run;
                    run += c;
                }
                base[i] = run;
            }
            __syncthreads();
            write_places<kRouteGroups>(a, tile0 + first, counts + wave * keys, key, rank);
        }
    }
}

size_t route_place_lds(int keys, bool sorted) {
    return (size_t)(1 + sorted + kRouteWaves) * keys * sizeof(int) +
           (sorted ? kRouteTile * (sizeof(int) + sizeof(uint16_t)) : 0);
}
static_assert((2 + kRouteWaves) * (kRouteMaxExperts + 1) * sizeof(int) + kRouteTile * 6 + 64 <= 65536, "LDS of a block");

int64_t route_tiles_per_block(int64_t pairs) {
    const int64_t tiles = (pairs + kRouteTile - 1) / kRouteTile;
    return std::max<int64_t>(1, (tiles + kRouteMaxBlocks - 1) / kRouteMaxBlocks);
}

int64_t route_blocks(int64_t pairs) {
    const int64_t span = route_tiles_per_block(pairs) * kRouteTile;
    return std::max<int64_t>(1, (pairs + span - 1) / span);
}

// Tiles sorted before they are stored, whole route: 4,194,304 pairs 49 -> 42 us
// with 256 experts, 40 -> 35 with 64, 32 -> 33 with 8; 1,048,576 pairs 24 -> 22,
// 19 -> 17 and 15 both ways, 500 experts 27 -> 25, 2048 experts 47 both ways;
// 524,288 pairs 18.4 -> 17.5 with 256 experts, 262,144 16.2 both ways, 65,536
// 15.2 -> 15.6.
bool route_sorted(int64_t pairs, int64_t E) { return pairs >= (int64_t(1) << 19) && E >= 64 && E <= 1024; }

// One launch up to 4,096 pairs: 5.7 to 7.9 us with 8 to 500 experts against
// 10.7 to 14.2 us for the three launches; at 8,192 pairs 10.8 to 16.5 against
// 11.3 to 14.5 us, at 16,384 14.7 to 22.9 against 11.6 to 14.9 us.
bool route_in_one_block(int64_t pairs, int64_t E) { return pairs <= 4096 && E + 1 <= 512; }

// --------------------------------------------------------------- exchange

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;
constexpr int64_t kStreamBytes = int64_t(128) << 20;     // half of the Infinity Cache

// How a call's accesses go: plain, non-temporal stores, non-temporal loads of
// what is read once as well.
enum Access { kPlain, kStores, kBoth };

template <int ACCESS, typename T>
__device__ inline Pack<T> load_once(const T *p, int64_t n) {
    if constexpr (ACCESS == kBoth) return load_pack_stream(p, n);
    else return load_pack(p, n);
}

template <int ACCESS, typename T>
__device__ inline void store_out(T *p, const Pack<T> &r, int64_t n) {
    if constexpr (ACCESS == kPlain) store_pack(p, r, n);
    else store_pack_stream(p, r, n);
}

// a = a * n + b for a position `b` behind the start of row `a` of rows of n, b < n + 2^13.
__device__ inline void carry(int64_t &row, uint32_t &col, uint32_t n) {
    if (n >= 8192) {
        if (col >= n) {
            col -= n;
            ++row;
        }
    } else {
        row += col / n;
        col %= n;
    }
}

// Row and column of element `at` of rows of n, for a position that is the
// same for the whole block.
__device__ inline void split(int64_t at, uint32_t n, int64_t *row, uint32_t *col) {
    if (at <= 0xffffffffLL) {
        *row = (uint32_t)at / n;
        *col = (uint32_t)at % n;
    } else {
        *row = at / n;
        *col = (uint32_t)(at % n);
    }
}

__device__ inline int64_t live_rows(const ExchangeArgs &a) {
    const int64_t kept = a.offsets[a.E], rows = a.T * a.k;
    return kept < 0 ? 0 : kept < rows ? kept : rows;
}

// Pair at place p, or -1 where the row is zero.
__device__ inline int pair_at(const ExchangeArgs &a, int64_t p, int64_t kept) {
    if (p >= kept) return -1;
    const int q = a.order[p];
    return q >= 0 && q < a.T * a.k ? q : -1;
}

// Element c of the output row that pair q fills (q < 0: zero).
template <typename T>
__device__ inline T dispatched(const ExchangeArgs &a, int q, uint32_t c) {
    if (q < 0) return (T)0.0f;
    const T v = ((const T *)a.rows)[(int64_t)((uint32_t)q / (uint32_t)a.k) * a.N + c];
    return a.weight ? (T)(load_weight<T>(a.weight, q, a.weight_fp32) * (float)v) : v;
}

// Pack number i of the output holds its elements [i * P - lead, i * P - lead
// + P): packs are aligned in memory, the first and last may be partial, and a
// pack may hold the end of one row and the start of the next.  A thread takes
// U packs, kThreads apart, so that their loads are in flight together.
template <typename T, int U, int ACCESS>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(ExchangeArgs a, int lead, int64_t blocks) {
    constexpr int P = kPack<T>;
    const int64_t kept = live_rows(a), rows = a.T * a.k, end = rows * a.N;
    const uint32_t N = (uint32_t)a.N, k = (uint32_t)a.k;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t first = b * (kThreads * U * P) - lead;    // below 0 in block 0 only
        int64_t p0;
        uint32_t c0;
        split(max(first, int64_t(0)), N, &p0, &c0);
        Pack<T> r[U], tail[U];
        int64_t at[U], p[U];
        uint32_t c[U];
        int q[U];
        bool whole[U], two[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at[u] = first + (threadIdx.x + u * kThreads) * P;
            p[u] = p0;
            c[u] = c0 + (uint32_t)(max(at[u], int64_t(0)) - max(first, int64_t(0)));
            if (at[u] < end) carry(p[u], c[u], N);
            q[u] = at[u] < end ? pair_at(a, p[u], kept) : -1;
            whole[u] = at[u] >= 0 && at[u] + P <= end && c[u] + P <= N;
            two[u] = false;
            r[u] = {};
            if (whole[u]) {
                if (q[u] >= 0) r[u] = load_pack((const T *)a.rows + (int64_t)((uint32_t)q[u] / k) * a.N + c[u]);
            } else if (at[u] >= 0 && at[u] + P <= end && N >= P && !a.weight) {
                // the end of one row and the start of the next: the packs of
                // x around them, where both lie inside x
                const int q1 = pair_at(a, p[u] + 1, kept);
                const int64_t from = (int64_t)((uint32_t)max(q[u], 0) / k) * a.N + c[u];
                const int64_t next = (int64_t)((uint32_t)max(q1, 0) / k) * a.N - (N - c[u]);
                two[u] = (q[u] < 0 || from + P <= a.T * a.N) && (q1 < 0 || next >= 0);
                tail[u] = {};
                if (two[u] && q[u] >= 0) r[u] = load_pack((const T *)a.rows + from);
                if (two[u] && q1 >= 0) tail[u] = load_pack((const T *)a.rows + next);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (whole[u]) {
                if (a.weight && q[u] >= 0) {
                    const float w = load_weight<T>(a.weight, q[u], a.weight_fp32);
#pragma unroll
                    for (int i = 0; i < P; ++i) r[u].v[i] = (T)(w * (float)r[u].v[i]);
                }
                store_out<ACCESS>((T *)a.out + at[u], r[u], P);
            } else if (two[u]) {
#pragma unroll
                for (uint32_t i = 0; i < P; ++i)
                    if (i >= N - c[u]) r[u].v[i] = tail[u].v[i];
                store_out<ACCESS>((T *)a.out + at[u], r[u], P);
            } else if (at[u] < end) {                               // the ends, and rows below a pack
                for (int64_t i = max(at[u], int64_t(0)); i < min(at[u] + P, end); ++i) {
                    ((T *)a.out)[i] = dispatched<T>(a, q[u], c[u]);
                    if (++c[u] == N) {
                        c[u] = 0;
                        q[u] = ++p[u] < rows ? pair_at(a, p[u], kept) : -1;
                    }
                }
            }
        }
    }
}

template <typename T, int ACCESS>
__global__ __launch_bounds__(kThreads) void combine_kernel(ExchangeArgs a, int64_t packs, int64_t total,
                                                           int64_t blocks) {
    const int64_t kept = live_rows(a);
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        if (b * kThreads + threadIdx.x >= total) continue;
        int64_t t;
        uint32_t v;
        split(b * kThreads, (uint32_t)packs, &t, &v);
        v += threadIdx.x;
        carry(t, v, (uint32_t)packs);
        const int64_t c = (int64_t)v * kPack<T>, n = a.N - c;
        float acc[kPack<T>] = {};
        for (int64_t j0 = 0; j0 < a.k; j0 += 4) {
            Pack<T> r[4];
            float w[4];
            bool live[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {           // the batch's loads go out before its first use
                const int64_t j = j0 + u;
                const int64_t p = j < a.k ? (int64_t)a.position[t * a.k + j] : -1;
                live[u] = p >= 0 && p < kept;
                w[u] = 1.0f;
                if (live[u]) {
                    r[u] = load_once<ACCESS>((const T *)a.rows + p * a.N + c, n);
                    if (a.weight) w[u] = load_weight<T>(a.weight, t * a.k + j, a.weight_fp32);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (live[u]) {
#pragma unroll
                    for (int i = 0; i < kPack<T>; ++i) acc[i] = fmaf(w[u], (float)r[u].v[i], acc[i]);
                }
        }
        Pack<T> o;
#pragma unroll
        for (int i = 0; i < kPack<T>; ++i) o.v[i] = (T)acc[i];
        store_out<ACCESS>((T *)a.out + t * a.N + c, o, n);
    }
}

// A group of G lanes takes one place: it walks its row and the row of dout
// once, writes the row's gradient and sums the dot product over the group.
template <typename T, int G, int ACCESS>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(ExchangeArgs a, int64_t packs) {
    const int64_t kept = live_rows(a), rows = a.T * a.k;
    const int lane = threadIdx.x % G;
    const Pack<T> zero = {};
    for (int64_t p0 = (int64_t)blockIdx.x * (kThreads / G); p0 < rows; p0 += (int64_t)gridDim.x * (kThreads / G)) {
        const int64_t p = p0 + threadIdx.x / G;
        int q = -1;
        bool live = false;
        float dot = 0.0f;
        if (p < rows) {
            q = a.order[p];
            if (q < 0 || q >= rows) q = -1;
            live = q >= 0 && p < kept;
            const float w = live && a.weight ? load_weight<T>(a.weight, q, a.weight_fp32) : 1.0f;
            const T *dout = (const T *)a.dout + (int64_t)((uint32_t)max(q, 0) / (uint32_t)a.k) * a.N;
            for (int64_t v = lane; v < packs; v += G) {
                const int64_t c = v * kPack<T>, n = a.N - c;
                Pack<T> o = zero;
                if (live) {
                    const Pack<T> d = load_pack(dout + c, n);
                    if (a.dweight) {
                        const Pack<T> r = load_once<ACCESS>((const T *)a.rows + p * a.N + c, n);
#pragma unroll
                        for (int i = 0; i < kPack<T>; ++i) dot = fmaf((float)r.v[i], (float)d.v[i], dot);
                    }
#pragma unroll
                    for (int i = 0; i < kPack<T>; ++i) o.v[i] = (T)(w * (float)d.v[i]);
                }
                if (a.drows) store_out<ACCESS>((T *)a.drows + p * a.N + c, o, n);
            }
        }
        if (a.dweight) {
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
            if (lane == 0 && q >= 0) store_weight<T>(a.dweight, q, a.weight_fp32, dot);
        }
    }
}

// Access of a call that moves `bytes`, and of its rows that are read once.
template <typename T>
int access_of(const ExchangeArgs &a, int64_t bytes) {
    if (bytes <= kStreamBytes) return kPlain;
    return a.N % kPack<T> == 0 && (uintptr_t)a.rows % 16 == 0 ? kBoth : kStores;
}

template <typename T>
hipError_t dispatch(const ExchangeArgs &a, hipStream_t s) {
    constexpr int P = kPack<T>;
    const int lead = (int)((uintptr_t)a.out % 16 / sizeof(T));
    const int64_t total = (a.T * a.k * a.N + lead + P - 1) / P;
    const bool plain = access_of<T>(a, (a.k + 1) * a.T * a.N * (int)sizeof(T)) == kPlain;
    // two packs to a thread once that still leaves every unit eight blocks
    const int per = total >= int64_t(256) * 8 * 2 * kThreads ? 2 : 1;
    const int64_t blocks = (total + kThreads * per - 1) / (kThreads * per);
    const unsigned grid = (unsigned)std::min(blocks, kMaxBlocks);
    if (per == 1) dispatch_kernel<T, 1, kPlain><<<grid, kThreads, 0, s>>>(a, lead, blocks);
    else if (plain) dispatch_kernel<T, 2, kPlain><<<grid, kThreads, 0, s>>>(a, lead, blocks);
    else dispatch_kernel<T, 2, kStores><<<grid, kThreads, 0, s>>>(a, lead, blocks);
    return hipGetLastError();
}

template <typename T>
hipError_t combine(const ExchangeArgs &a, hipStream_t s) {
    const int64_t packs = (a.N + kPack<T> - 1) / kPack<T>, total = a.T * packs;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)std::min(blocks, kMaxBlocks);
    const int access = access_of<T>(a, (a.k + 1) * a.T * a.N * (int)sizeof(T));
    if (access == kPlain) combine_kernel<T, kPlain><<<grid, kThreads, 0, s>>>(a, packs, total, blocks);
    else if (access == kStores) combine_kernel<T, kStores><<<grid, kThreads, 0, s>>>(a, packs, total, blocks);
    else combine_kernel<T, kBoth><<<grid, kThreads, 0, s>>>(a, packs, total, blocks);
    return hipGetLastError();
}

template <typename T, int G>
hipError_t combine_backward_groups(const ExchangeArgs &a, int64_t packs, hipStream_t s) {
    const int64_t rows = a.T * a.k, blocks = (rows + kThreads / G - 1) / (kThreads / G);
    const unsigned grid = (unsigned)std::min(blocks, kMaxBlocks);
    const int access = access_of<T>(a, (2 * a.k + 1) * a.T * a.N * (int)sizeof(T));
    if (access == kPlain) combine_backward_kernel<T, G, kPlain><<<grid, kThreads, 0, s>>>(a, packs);
    else if (access == kStores) combine_backward_kernel<T, G, kStores><<<grid, kThreads, 0, s>>>(a, packs);
    else combine_backward_kernel<T, G, kBoth><<<grid, kThreads, 0, s>>>(a, packs);
    return hipGetLastError();
}

template <typename T>
hipError_t combine_backward(const ExchangeArgs &a, hipStream_t s) {
    const int64_t packs = (a.N + kPack<T> - 1) / kPack<T>;
    if (packs <= 4) return combine_backward_groups<T, 4>(a, packs, s);
    if (packs <= 16) return combine_backward_groups<T, 16>(a, packs, s);
    return combine_backward_groups<T, 64>(a, packs, s);
}

}  // namespace

int64_t route_workspace_ints(int64_t pairs, int64_t E) {
    if (route_in_one_block(pairs, E)) return 0;
    return (E + 1) * (route_blocks(pairs) + 1);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t s) {
    const int keys = a.E + 1;
    int bits = 0;
    while ((1 << bits) < keys) ++bits;
    if (route_in_one_block(a.pairs, a.E)) {
        const size_t lds = (size_t)16 * keys * sizeof(int);
        if (a.pairs <= 1024) route_one_kernel<1><<<1, 1024, lds, s>>>(a, bits);
        else route_one_kernel<4><<<1, 1024, lds, s>>>(a, bits);
        return hipGetLastError();
    }
    const int64_t nblocks = route_blocks(a.pairs), per = route_tiles_per_block(a.pairs);
    int *hist = a.workspace, *total_of = a.workspace + (int64_t)keys * nblocks;
    route_count_kernel<<<(unsigned)nblocks, kRouteThreads, keys * sizeof(int), s>>>(a, per);
    route_scan_kernel<<<(unsigned)keys, kRouteThreads, 0, s>>>(hist, (int)nblocks, total_of);
    const bool sorted = route_sorted(a.pairs, a.E);
    const size_t lds = route_place_lds(keys, sorted);
    if (sorted) route_place_kernel<true><<<(unsigned)nblocks, kRouteThreads, lds, s>>>(a, hist, total_of, bits, per);
    else route_place_kernel<false><<<(unsigned)nblocks, kRouteThreads, lds, s>>>(a, hist, total_of, bits, per);
    return hipGetLastError();
}

hipError_t launch_dispatch(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return dispatch<float>(a, s);
    if (type == SPMM_BF16) return dispatch<__bf16>(a, s);
    return dispatch<_Float16>(a, s);
}

hipError_t launch_combine(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return combine<float>(a, s);
    if (type == SPMM_BF16) return combine<__bf16>(a, s);
    return combine<_Float16>(a, s);
}

hipError_t launch_combine_backward(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return combine_backward<float>(a, s);
    if (type == SPMM_BF16) return combine_backward<__bf16>(a, s);
    return combine_backward<_Float16>(a, s);
}

}  // namespace gspmm
