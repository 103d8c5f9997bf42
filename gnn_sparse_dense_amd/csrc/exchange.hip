// The routed exchange: rows sorted by expert, copied into that order, and the
// experts' rows summed back with weights, with the gradients of both.
//
//  * Route.  The pairs p = t * k + j are sorted by expert, stably; pairs whose
//    expert is outside [0, E) come last.  A counting sort: a pair's place is
//    (pairs of smaller experts) + (pairs of its expert in earlier blocks and
//    waves) + (its rank inside its wave).  The rank comes from ballots: the
//    lanes of a wave that hold the same key are found with one ballot per key
//    bit, so equal keys keep their order and no atomic decides a place.
//  * Dispatch: out[position[t, j]] = x[t].  Rows are walked by source, so
//    every row of x is read once and written k times.
//  * Combine: out[t] = sum_j weight[t, j] * rows[position[t, j]], j ascending,
//    one fused multiply-add per term.  With no weights it is dispatch's
//    gradient.
//  * Combine's gradients: drows[position[t, j]] = weight[t, j] * dout[t] and
//    dweight[t, j] = <rows[position[t, j]], dout[t]>, one pass over both.
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
constexpr int kRouteGroups = 16;
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
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kRouteThreads) atomicAdd(&lds[route_key(a.expert[p], a.E)], 1);
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

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a, const int *hist, const int *total_of,
                                                                    int bits, int64_t tiles_per_block) {
    extern __shared__ int lds[];                     // base[keys], count[kRouteWaves][keys]
    __shared__ int sh[kRouteWaves];
    const int keys = a.E + 1, wave = threadIdx.x / kWave;
    int *base = lds, *counts = lds + keys;
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
        const int64_t first = tile0 + (int64_t)wave * kRouteGroups * kWave;
        rank_in_wave<kRouteGroups>(a, first, bits, counts + wave * keys, key, rank);
        __syncthreads();
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
        write_places<kRouteGroups>(a, first, counts + wave * keys, key, rank);
    }
}

int64_t route_tiles_per_block(int64_t pairs) {
    const int64_t tiles = (pairs + kRouteTile - 1) / kRouteTile;
    return std::max<int64_t>(1, (tiles + kRouteMaxBlocks - 1) / kRouteMaxBlocks);
}

int64_t route_blocks(int64_t pairs) {
    const int64_t span = route_tiles_per_block(pairs) * kRouteTile;
    return std::max<int64_t>(1, (pairs + span - 1) / span);
}

bool route_in_one_block(int64_t pairs, int64_t E) { return pairs <= 16 * 1024 && E + 1 <= 512; }

// --------------------------------------------------------------- exchange

constexpr int kThreads = 256;

// A launch's work as a flat list of (row, pack) items, 256 to a block.
struct Items {
    int64_t packs;      // packs of a row
    int64_t total;      // rows * packs
};

__host__ __device__ inline int64_t packs_of(int64_t N, int pack) { return (N + pack - 1) / pack; }

// Row and pack of the thread's item.  The block's first item is split with
// one division in 32 bits where the launch fits them, the thread's with a
// comparison or a 32-bit division.
__device__ inline bool item_of(int64_t block, int64_t packs, int64_t total, int64_t *row, int64_t *pack) {
    const int64_t b0 = block * kThreads;
    int64_t r, v;
    if (total <= 0xffffffffLL) {
        r = (uint32_t)b0 / (uint32_t)packs;
        v = (uint32_t)b0 % (uint32_t)packs;
    } else {
        r = b0 / packs;
        v = b0 % packs;
    }
    v += threadIdx.x;
    if (packs >= kThreads) {
        if (v >= packs) {
            v -= packs;
            ++r;
        }
    } else {
        r += (uint32_t)v / (uint32_t)packs;
        v = (uint32_t)v % (uint32_t)packs;
    }
    *row = r;
    *pack = v;
    return b0 + threadIdx.x < total;
}

__device__ inline int64_t live_rows(const ExchangeArgs &a) {
    const int64_t kept = a.offsets[a.E], rows = a.T * a.k;
    return kept < 0 ? 0 : kept < rows ? kept : rows;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(ExchangeArgs a, int64_t packs, int64_t total,
                                                            int64_t blocks) {
    const int64_t kept = live_rows(a), rows = a.T * a.k;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        int64_t t, v;
        if (!item_of(b, packs, total, &t, &v)) continue;
        const int64_t c = v * kPack<T>, n = a.N - c;
        const Pack<T> x = load_pack((const T *)a.rows + t * a.N + c, n);
        const Pack<T> zero = {};
        for (int64_t j = 0; j < a.k; ++j) {
            const int64_t p = a.position[t * a.k + j];
            if (p < 0 || p >= rows) continue;
            Pack<T> r = x;
            if (a.weight) {
                const float w = load_weight<T>(a.weight, t * a.k + j, a.weight_fp32);
#pragma unroll
                for (int i = 0; i < kPack<T>; ++i) r.v[i] = (T)(w * (float)x.v[i]);
            }
            store_pack((T *)a.out + p * a.N + c, p < kept ? r : zero, n);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void combine_kernel(ExchangeArgs a, int64_t packs, int64_t total,
                                                           int64_t blocks) {
    const int64_t kept = live_rows(a);
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        int64_t t, v;
        if (!item_of(b, packs, total, &t, &v)) continue;
        const int64_t c = v * kPack<T>, n = a.N - c;
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
                    r[u] = load_pack((const T *)a.rows + p * a.N + c, n);
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
        store_pack((T *)a.out + t * a.N + c, o, n);
    }
}

// A group of G lanes takes one pair: it walks the row of dout and the pair's
// row once, writes the row's gradient and sums the dot product over the group.
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(ExchangeArgs a, int64_t packs, int64_t tasks) {
    const int64_t kept = live_rows(a), rows = a.T * a.k;
    const int lane = threadIdx.x % G;
    const Pack<T> zero = {};
    for (int64_t task0 = (int64_t)blockIdx.x * (kThreads / G); task0 < tasks;
         task0 += (int64_t)gridDim.x * (kThreads / G)) {
        const int64_t task = task0 + threadIdx.x / G;
        float dot = 0.0f;
        if (task < tasks) {
            const int64_t t = task / a.k, p = a.position[task];
            const bool live = p >= 0 && p < kept;
            const float w = a.weight ? load_weight<T>(a.weight, task, a.weight_fp32) : 1.0f;
            for (int64_t v = lane; v < packs; v += G) {
                const int64_t c = v * kPack<T>, n = a.N - c;
                if (live) {
                    const Pack<T> d = load_pack((const T *)a.dout + t * a.N + c, n);
                    if (a.dweight) {
                        const Pack<T> r = load_pack((const T *)a.rows + p * a.N + c, n);
#pragma unroll
                        for (int i = 0; i < kPack<T>; ++i) dot = fmaf((float)r.v[i], (float)d.v[i], dot);
                    }
                    if (a.drows) {
                        Pack<T> o;
#pragma unroll
                        for (int i = 0; i < kPack<T>; ++i) o.v[i] = (T)(w * (float)d.v[i]);
                        store_pack((T *)a.drows + p * a.N + c, o, n);
                    }
                } else if (a.drows && p >= 0 && p < rows) {
                    store_pack((T *)a.drows + p * a.N + c, zero, n);
                }
            }
        }
        if (a.dweight) {
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) dot += __shfl_xor(dot, o, kWave);
            if (lane == 0 && task < tasks) store_weight<T>(a.dweight, task, a.weight_fp32, dot);
        }
    }
}

constexpr int64_t kMaxBlocks = 1 << 20;

template <typename T>
hipError_t flat(void (*kernel)(ExchangeArgs, int64_t, int64_t, int64_t), const ExchangeArgs &a, hipStream_t s) {
    const int64_t packs = packs_of(a.N, kPack<T>), total = a.T * packs;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    if (blocks == 0) return hipSuccess;
    kernel<<<(unsigned)std::min(blocks, kMaxBlocks), kThreads, 0, s>>>(a, packs, total, blocks);
    return hipGetLastError();
}

template <typename T, int G>
hipError_t grouped(const ExchangeArgs &a, hipStream_t s) {
    const int64_t tasks = a.T * a.k, blocks = (tasks + kThreads / G - 1) / (kThreads / G);
    if (blocks == 0) return hipSuccess;
    combine_backward_kernel<T, G><<<(unsigned)std::min(blocks, kMaxBlocks), kThreads, 0, s>>>(
        a, packs_of(a.N, kPack<T>), tasks);
    return hipGetLastError();
}

template <typename T>
hipError_t combine_backward(const ExchangeArgs &a, hipStream_t s) {
    const int64_t packs = packs_of(a.N, kPack<T>);
    if (packs <= 4) return grouped<T, 4>(a, s);
    if (packs <= 16) return grouped<T, 16>(a, s);
    return grouped<T, 64>(a, s);
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
        else if (a.pairs <= 4096) route_one_kernel<4><<<1, 1024, lds, s>>>(a, bits);
        else route_one_kernel<16><<<1, 1024, lds, s>>>(a, bits);
        return hipGetLastError();
    }
    const int64_t nblocks = route_blocks(a.pairs), per = route_tiles_per_block(a.pairs);
    int *hist = a.workspace, *total_of = a.workspace + (int64_t)keys * nblocks;
    route_count_kernel<<<(unsigned)nblocks, kRouteThreads, keys * sizeof(int), s>>>(a, per);
    route_scan_kernel<<<(unsigned)keys, kRouteThreads, 0, s>>>(hist, (int)nblocks, total_of);
    route_place_kernel<<<(unsigned)nblocks, kRouteThreads, (size_t)(1 + kRouteWaves) * keys * sizeof(int), s>>>(
        a, hist, total_of, bits, per);
    return hipGetLastError();
}

hipError_t launch_dispatch(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return flat<float>(dispatch_kernel<float>, a, s);
    if (type == SPMM_BF16) return flat<__bf16>(dispatch_kernel<__bf16>, a, s);
    return flat<_Float16>(dispatch_kernel<_Float16>, a, s);
}

hipError_t launch_combine(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return flat<float>(combine_kernel<float>, a, s);
    if (type == SPMM_BF16) return flat<__bf16>(combine_kernel<__bf16>, a, s);
    return flat<_Float16>(combine_kernel<_Float16>, a, s);
}

hipError_t launch_combine_backward(const ExchangeArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return combine_backward<float>(a, s);
    if (type == SPMM_BF16) return combine_backward<__bf16>(a, s);
    return combine_backward<_Float16>(a, s);
}

}  // namespace gspmm
