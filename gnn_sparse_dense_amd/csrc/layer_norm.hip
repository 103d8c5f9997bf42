// Layer norm over the rows of [R, N], forward and backward.
//
//   mean = sum(x) / N, var = sum((x - mean)^2) / N, rstd = 1 / sqrt(var + eps)
//   u = (x - mean) * rstd,  y = u * weight + bias
//   g = dy * weight,  dx = rstd * (g - mean(g) - u * mean(g * u))
//   dweight = sum over rows of dy * u,  dbias = sum over rows of dy
//
// A row is read once into the registers of a group of G lanes (NV packs of 16
// bytes per lane), the mean and then the centred squares are summed there,
// and the row is written once: 2 R N elements forward, 3 R N backward, which
// is what bounds both.  The next row of the group is loaded before the
// current one is summed.  Groups of more than a wave join their waves' means
// and centred squares (Chan, Golub and LeVeque's pairwise rule) behind one
// barrier.  A group keeps its columns
// while it walks rows, so the weights stay in registers and the backward pass
// adds dy * u and dy of its columns in fp32 registers; at its end a block adds
// its groups' sums and writes one partial row per gradient, and a second
// kernel adds the partial rows in block order (no atomics).  Rows too long for
// registers are read once for each sum instead.
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kWave = 64;
constexpr int64_t kStreamBytes = int64_t(128) << 20;     // half of the Infinity Cache

template <int CTRL>
__device__ inline float add_lane(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf,
                                                                     false));
}

__device__ inline float from_lane(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Sum over aligned groups of LANES lanes, the same bits in every lane: within
// quads, quads of 8, halves of 16, then rows of 16 through scalar registers.
template <int LANES>
__device__ inline float lanes_sum(float v) {
    v = add_lane<0xB1>(v);
    v = add_lane<0x4E>(v);
    if constexpr (LANES >= 8) v = add_lane<0x141>(v);
    if constexpr (LANES >= 16) v = add_lane<0x140>(v);
    if constexpr (LANES >= 32) {
        const float low = from_lane(v, 0) + from_lane(v, 16), high = from_lane(v, 32) + from_lane(v, 48);
        if constexpr (LANES == 32) v = (threadIdx.x & 32) ? high : low;
        else v = low + high;
    }
    return v;
}

// Sums of NS values over the group of G lanes, in every lane.  Groups of more
// than a wave hand the waves' sums over in sh, NS floats for each wave of the
// block; the caller alternates between two of them so that one barrier is
// enough.
template <int G, int NS>
__device__ inline void group_sum(float (&v)[NS], float *sh) {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = lanes_sum<(G < kWave ? G : kWave)>(v[i]);
    if constexpr (G > kWave) {
        constexpr int kWaves = G / kWave;
        const int wave = threadIdx.x / kWave, base = wave / kWaves * kWaves;
        if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) sh[wave * NS + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) t += sh[(base + w) * NS + i];
            v[i] = t;
        }
    }
}

template <int G>
constexpr int kBlockOf = G > 256 ? G : 256;

// The lane's columns: NV packs of P, pack q from column (q G + lane) P.  A
// pack that would end behind the row is moved back to end there, and owns
// only what its neighbour does not hold (skip elements less; none when it
// begins behind the row), so that every load is whole and inside the row.
// NARROW: rows of fewer than P elements, all owned by lane 0.
template <int G, int NV, int P, bool NARROW>
struct Columns {
    int at[NV], skip[NV];
    unsigned ragged;        // packs that some lane of the wave does not own whole
    int N;

    __device__ inline Columns(int64_t n) {
        const int lane = threadIdx.x % G;
        N = (int)n;
        ragged = 0;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t c = (int64_t)(q * G + lane) * P;
            at[q] = NARROW ? 0 : (int)min(c, n - P);
            skip[q] = NARROW ? (lane ? P : 0) : (int)min(int64_t(P), c - at[q]);
            if (NARROW || __ballot(skip[q] > 0)) ragged |= 1u << q;
        }
    }

    // f(i, owned) for the elements of pack q
    template <typename F>
    __device__ inline void each(int q, F f) const {
        if (ragged >> q & 1) {
#pragma unroll
            for (int i = 0; i < P; ++i) f(i, i >= skip[q] && (!NARROW || i < N));
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) f(i, true);
        }
    }

    template <typename T>
    __device__ inline Pack<T> load(const T *row, int q) const {
        if constexpr (NARROW) return load_pack(row, N);
        else return load_pack(row + at[q]);
    }

    template <typename T>
    __device__ inline void store(T *row, int q, const Pack<T> &v, bool stream) const {
        if (!(ragged >> q & 1) || (!NARROW && skip[q] == 0)) {
            if (stream) store_pack_stream(row + at[q], v, P);
            else store_pack(row + at[q], v, P);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (i >= skip[q] && (!NARROW || i < N)) row[at[q] + i] = v.v[i];
        }
    }
};

// The lane's weights of one pack, in the registers as they are stored:
// converted to fp32 where they are used, in every row, since the converted
// values would take twice the registers.
template <typename W, int P>
struct Weights {
    static constexpr int kWords = P * (int)sizeof(W) / 4;
    int word[kWords];

    template <bool NARROW>
    __device__ inline void load(const void *p, int at, int N, float none) {
        W v[P];
        if (p && !NARROW) {
            __builtin_memcpy(v, static_cast<const W *>(p) + at, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = p && i < N ? static_cast<const W *>(p)[i] : (W)none;
        }
        __builtin_memcpy(word, v, sizeof(word));
    }

    __device__ inline void get(float (&to)[P]) {
        if constexpr (sizeof(W) < 4)
#pragma unroll
            for (int &w : word) asm volatile("" : "+v"(w));      // not moved out of the loop over rows
        W v[P];
        __builtin_memcpy(v, word, sizeof(word));
#pragma unroll
        for (int i = 0; i < P; ++i) to[i] = (float)v[i];
    }
};

// Keeps 16-bit packs as they were loaded: without it their fp32 values stay in
// registers from one pass over the row to the next, twice as many.
template <typename T, int NV>
__device__ inline void keep_packed(Pack<T> (&x)[NV]) {
    if constexpr (sizeof(T) == 2)
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            int word[4];
            __builtin_memcpy(word, &x[q], sizeof(word));
#pragma unroll
            for (int &w : word) asm volatile("" : "+v"(w));
            __builtin_memcpy(&x[q], word, sizeof(word));
        }
}

template <typename T, typename W, int G, int NV, bool NARROW = false>
__global__ __launch_bounds__(kBlockOf<G>) void norm_kernel(NormArgs a, bool stream) {
    constexpr int P = kPack<T>, kRows = kBlockOf<G> / G, kWaves = kBlockOf<G> / kWave, kGroupWaves = G / kWave;
    constexpr int kLanes = G < kWave ? G : kWave;
    constexpr bool kAhead = G * NV < 4096;           // registers for the weights and a second row
    __shared__ float sh[2][2 * (G > kWave ? kWaves : 1)];
    const Columns<G, NV, P, NARROW> cols(a.N);
    const float inv_n = 1.0f / (float)a.N;
    Weights<W, P> weight[NV], bias[NV];
    Pack<T> x[NV], ahead[NV];
    const int64_t first = (int64_t)blockIdx.x * kRows, stride = (int64_t)gridDim.x * kRows;
    const int group = threadIdx.x / G;
    auto load = [&](int64_t r, Pack<T>(&to)[NV]) {               // a row behind the last: the last again
#pragma unroll
        for (int q = 0; q < NV; ++q) to[q] = cols.load((const T *)a.x + min(r, a.R - 1) * a.N, q);
    };
    if constexpr (kAhead) load(first + group, x);
    auto load_weights = [&](int q) {
        weight[q].template load<NARROW>(a.weight, cols.at[q], cols.N, 1.0f);
        bias[q].template load<NARROW>(a.bias, cols.at[q], cols.N, 0.0f);
    };
#pragma unroll
    for (int q = 0; q < NV; ++q)
        if constexpr (kAhead) load_weights(q);
    // elements of the row that wave w of the group holds
    auto wave_elements = [&](int w) {
        int64_t n = 0;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            n += max(int64_t(0), min(int64_t(kWave * P), a.N - (int64_t)(q * G + w * kWave) * P));
        return (float)n;
    };
    const float mine = G > kWave ? wave_elements(threadIdx.x % G / kWave) : 0.0f;
    // every group of a block takes the same number of turns (the barriers)
    int turn = 0;
    for (int64_t r0 = first; r0 < a.R; r0 += stride, turn ^= 1) {
        const int64_t r = r0 + group;
        if constexpr (kAhead) load(r + stride, ahead);
        else load(r, x);
        float s = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int q = 0; q < NV; ++q) cols.each(q, [&](int i, bool own) { s += own ? (float)x[q].v[i] : 0.0f; });
        s = lanes_sum<kLanes>(s);
        keep_packed(x);
        float mean = G <= kWave ? s * inv_n : mine > 0.0f ? s / mine : 0.0f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            cols.each(q, [&](int i, bool own) {
                const float d = own ? (float)x[q].v[i] - mean : 0.0f;
                m2 = fmaf(d, d, m2);
            });
        m2 = lanes_sum<kLanes>(m2);
        keep_packed(x);
        if constexpr (G > kWave) {
            const int wave = threadIdx.x / kWave, base = wave / kGroupWaves * kGroupWaves;
            if ((threadIdx.x & (kWave - 1)) == 0) {
                sh[turn][2 * wave] = s;
                sh[turn][2 * wave + 1] = m2;
            }
            __syncthreads();
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kGroupWaves; ++w) sum += sh[turn][2 * (base + w)];
            mean = sum * inv_n;
            m2 = 0.0f;
#pragma unroll
            for (int w = 0; w < kGroupWaves; ++w) {
                const float n = wave_elements(w), d = n > 0.0f ? sh[turn][2 * (base + w)] / n - mean : 0.0f;
                m2 += fmaf(n * d, d, sh[turn][2 * (base + w) + 1]);
            }
        }
        const float rstd = 1.0f / sqrtf(m2 * inv_n + a.eps);
        if (r < a.R) {
            if (threadIdx.x % G == 0 && a.mean) {
                a.mean[r] = mean;
                a.rstd[r] = rstd;
            }
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                Pack<T> y;
                float w[P], b[P];
                if constexpr (!kAhead) load_weights(q);
                weight[q].get(w);
                bias[q].get(b);
#pragma unroll
                for (int i = 0; i < P; ++i) y.v[i] = (T)fmaf(((float)x[q].v[i] - mean) * rstd, w[i], b[i]);
                cols.store((T *)a.y + r * a.N, q, y, stream);
            }
        }
        if constexpr (kAhead)
#pragma unroll
            for (int q = 0; q < NV; ++q) x[q] = ahead[q];
    }
}

// Rows too long for registers.  whole(c) for the packs of a row, `each` lane
// of the block its own, four in flight; one(c) for the elements behind the
// last whole pack.
constexpr int kLongLanes = 1024;

template <int P, typename F, typename H>
__device__ inline void walk_row(int64_t N, F whole, H one) {
    const int64_t end = N / P * P;
#pragma unroll 4
    for (int64_t c = (int64_t)threadIdx.x * P; c < end; c += kLongLanes * P) whole(c);
    for (int64_t c = end + threadIdx.x; c < N; c += kLongLanes) one(c);
}

// One block per row, three reads.
template <typename T>
__global__ __launch_bounds__(kLongLanes) void norm_long_kernel(NormArgs a) {
    constexpr int P = kPack<T>;
    __shared__ float sh[2][kLongLanes / kWave];
    const float inv_n = 1.0f / (float)a.N;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.N;
        T *y = (T *)a.y + r * a.N;
        float s[1] = {0.0f};
        walk_row<P>(
            a.N,
            [&](int64_t c) {
                const Pack<T> v = load_pack(x + c);
#pragma unroll
                for (int i = 0; i < P; ++i) s[0] += (float)v.v[i];
            },
            [&](int64_t c) { s[0] += (float)x[c]; });
        group_sum<kLongLanes, 1>(s, sh[0]);
        const float mean = s[0] * inv_n;
        s[0] = 0.0f;
        auto square = [&](float v) { s[0] = fmaf(v - mean, v - mean, s[0]); };
        walk_row<P>(
            a.N,
            [&](int64_t c) {
                const Pack<T> v = load_pack(x + c);
#pragma unroll
                for (int i = 0; i < P; ++i) square((float)v.v[i]);
            },
            [&](int64_t c) { square((float)x[c]); });
        group_sum<kLongLanes, 1>(s, sh[1]);
        const float rstd = 1.0f / sqrtf(s[0] * inv_n + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        auto out = [&](float v, int64_t c) {
            const float w = a.weight ? load_weight<T>(a.weight, c, a.weight_fp32) : 1.0f;
            const float b = a.bias ? load_weight<T>(a.bias, c, a.weight_fp32) : 0.0f;
            return (T)fmaf((v - mean) * rstd, w, b);
        };
        walk_row<P>(
            a.N,
            [&](int64_t c) {
                Pack<T> v = load_pack(x + c);
#pragma unroll
                for (int i = 0; i < P; ++i) v.v[i] = out((float)v.v[i], c + i);
                store_pack(y + c, v, P);
            },
            [&](int64_t c) { y[c] = out((float)x[c], c); });
    }
}

// partial: [gridDim.x][2][N] (dweight, dbias), written when a.partial is set.
template <typename T, typename W, int G, int NV, bool NARROW = false>
__global__ __launch_bounds__(kBlockOf<G>) void norm_backward_kernel(NormArgs a, bool stream) {
    constexpr int P = kPack<T>, kRows = kBlockOf<G> / G, kWaves = kBlockOf<G> / kWave;
    __shared__ float sh[2][2 * (G > kWave ? kWaves : 1)];
    const Columns<G, NV, P, NARROW> cols(a.N);
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const float inv_n = 1.0f / (float)a.N;
    Weights<W, P> weight[NV];
    float dw[NV][P] = {}, db[NV][P] = {};
    Pack<T> x[NV] = {}, d[NV] = {}, x_ahead[NV] = {}, d_ahead[NV] = {};
    float mean = 0.0f, rstd = 0.0f, mean_ahead = 0.0f, rstd_ahead = 0.0f;
    const int64_t first = (int64_t)blockIdx.x * kRows, stride = (int64_t)gridDim.x * kRows;
    auto load = [&](int64_t r, Pack<T>(&tx)[NV], Pack<T>(&td)[NV], float &m, float &s) {
        r = min(r, a.R - 1);                         // a row behind the last: the last again
        m = a.mean[r];
        s = a.rstd[r];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            tx[q] = cols.load((const T *)a.x + r * a.N, q);
            td[q] = cols.load((const T *)a.dy + r * a.N, q);
        }
    };
    if (a.R > 0) load(first + group, x, d, mean, rstd);
#pragma unroll
    for (int q = 0; q < NV; ++q) weight[q].template load<NARROW>(a.weight, cols.at[q], cols.N, 1.0f);
    int turn = 0;
    for (int64_t r0 = first; r0 < a.R; r0 += stride, turn ^= 1) {
        const int64_t r = r0 + group;
        const bool live = r < a.R;
        load(r + stride, x_ahead, d_ahead, mean_ahead, rstd_ahead);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            float w[P];
            weight[q].get(w);
            cols.each(q, [&](int i, bool own) {
                const bool in = own && live;
                const float u = in ? ((float)x[q].v[i] - mean) * rstd : 0.0f;
                const float dy = in ? (float)d[q].v[i] : 0.0f, g = dy * w[i];
                s[0] += g;
                s[1] = fmaf(g, u, s[1]);
                dw[q][i] = fmaf(dy, u, dw[q][i]);
                db[q][i] += dy;
            });
        }
        if (a.dx) {                                  // the same for every lane
            group_sum<G, 2>(s, sh[turn]);
            keep_packed(x);
            keep_packed(d);
            const float mg = s[0] * inv_n, mgu = s[1] * inv_n;
            if (live)
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    Pack<T> o;
                    float w[P];
                    weight[q].get(w);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float u = ((float)x[q].v[i] - mean) * rstd, g = (float)d[q].v[i] * w[i];
                        o.v[i] = (T)(rstd * (g - mg - u * mgu));
                    }
                    cols.store((T *)a.dx + r * a.N, q, o, stream);
                }
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            x[q] = x_ahead[q];
            d[q] = d_ahead[q];
        }
        mean = mean_ahead;
        rstd = rstd_ahead;
    }
    if (!a.partial) return;
    // the block's groups: lanes of a wave first, then its waves
    if constexpr (G < kWave) {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int o = G; o < kWave; o <<= 1) {
                    dw[q][i] += __shfl_xor(dw[q][i], o, kWave);
                    db[q][i] += __shfl_xor(db[q][i], o, kWave);
                }
    }
    float *out = a.partial + (int64_t)blockIdx.x * 2 * a.N;
    if constexpr (kRows > 1) {
        constexpr int kSets = G < kWave ? kWaves : kRows, kLanes = G;
        __shared__ float acc[kSets][2][NV][P][kLanes];
        const int set = G < kWave ? threadIdx.x / kWave : group;
        if (G >= kWave || (threadIdx.x & (kWave - 1)) < kLanes)
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    acc[set][0][q][i][lane] = dw[q][i];
                    acc[set][1][q][i][lane] = db[q][i];
                }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * NV * P * kLanes; i += kBlockOf<G>) {
            const int l = i % kLanes, e = i / kLanes % P, q = i / (kLanes * P) % NV, which = i / (kLanes * P * NV);
            const int64_t c = (int64_t)(q * G + l) * P, at = NARROW ? 0 : min(c, a.N - P);
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kSets; ++w) t += acc[w][which][q][e][l];
            if (NARROW ? c + e < a.N : e >= c - at) out[which * a.N + at + e] = t;
        }
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q)
            cols.each(q, [&](int i, bool own) {
                if (own) {
                    out[cols.at[q] + i] = dw[q][i];
                    out[a.N + cols.at[q] + i] = db[q][i];
                }
            });
    }
}

// Rows too long for registers: dx with two reads of the row.
template <typename T>
__global__ __launch_bounds__(kLongLanes) void norm_backward_long_kernel(NormArgs a) {
    constexpr int P = kPack<T>;
    __shared__ float sh[2][2 * kLongLanes / kWave];
    const float inv_n = 1.0f / (float)a.N;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        const T *x = (const T *)a.x + r * a.N, *dy = (const T *)a.dy + r * a.N;
        T *dx = (T *)a.dx + r * a.N;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s[2] = {0.0f, 0.0f};
        auto weighted = [&](float d, int64_t c) {
            return a.weight ? d * load_weight<T>(a.weight, c, a.weight_fp32) : d;
        };
        auto sums = [&](float v, float d, int64_t c) {
            const float g = weighted(d, c);
            s[0] += g;
            s[1] = fmaf(g, (v - mean) * rstd, s[1]);
        };
        walk_row<P>(
            a.N,
            [&](int64_t c) {
                const Pack<T> v = load_pack(x + c), d = load_pack(dy + c);
#pragma unroll
                for (int i = 0; i < P; ++i) sums((float)v.v[i], (float)d.v[i], c + i);
            },
            [&](int64_t c) { sums((float)x[c], (float)dy[c], c); });
        group_sum<kLongLanes, 2>(s, sh[turn]);
        const float mg = s[0] * inv_n, mgu = s[1] * inv_n;
        auto out = [&](float v, float d, int64_t c) {
            return (T)(rstd * (weighted(d, c) - mg - (v - mean) * rstd * mgu));
        };
        walk_row<P>(
            a.N,
            [&](int64_t c) {
                const Pack<T> v = load_pack(x + c), d = load_pack(dy + c);
                Pack<T> o;
#pragma unroll
                for (int i = 0; i < P; ++i) o.v[i] = out((float)v.v[i], (float)d.v[i], c + i);
                store_pack(dx + c, o, P);
            },
            [&](int64_t c) { dx[c] = out((float)x[c], (float)dy[c], c); });
    }
}

// ... and the weights' gradients by columns: block (columns, chunk of rows).
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs a, int64_t rows_per_chunk) {
    constexpr int P = kPack<T>;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * P;
    if (c >= a.N) return;
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_chunk, r1 = min(a.R, r0 + rows_per_chunk);
    float dw[P] = {}, db[P] = {};
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        const Pack<T> v = load_pack((const T *)a.x + r * a.N + c, a.N - c);
        const Pack<T> d = load_pack((const T *)a.dy + r * a.N + c, a.N - c);
        const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            dw[i] = fmaf((float)d.v[i], ((float)v.v[i] - mean) * rstd, dw[i]);
            db[i] += (float)d.v[i];
        }
    }
    float *out = a.partial + (int64_t)blockIdx.y * 2 * a.N;
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (c + i < a.N) {
            out[c + i] = dw[i];
            out[a.N + c + i] = db[i];
        }
}

// dweight / dbias: the partial rows added in order, each thread a strided
// part of them, the parts added in order.  16 columns of [2][N] per block, so
// that narrow rows still give several blocks.
constexpr int kFoldColumns = 16, kFoldParts = 64;

template <typename T>
__global__ __launch_bounds__(kFoldColumns *kFoldParts) void norm_fold_kernel(NormArgs a, int64_t parts) {
    __shared__ float sh[kFoldParts][kFoldColumns];
    const int col = threadIdx.x % kFoldColumns, part = threadIdx.x / kFoldColumns;
    const int64_t c = (int64_t)blockIdx.x * kFoldColumns + col;      // over [2][N]
    float t = 0.0f;
    if (c < 2 * a.N)
#pragma unroll 8
        for (int64_t p = part; p < parts; p += kFoldParts) t += a.partial[p * 2 * a.N + c];
    sh[part][col] = t;
    __syncthreads();
    if (part != 0 || c >= 2 * a.N) return;
#pragma unroll
    for (int p = 1; p < kFoldParts; ++p) t += sh[p][col];
    void *out = c < a.N ? a.dweight : a.dbias;
    if (out) store_weight<T>(out, c < a.N ? c : c - a.N, a.weight_fp32, t);
}

// ---- shapes ----

// Lanes of a row's group and packs per lane; 0 lanes: too long for registers.
// Two packs per lane: with the weights, the row ahead and (backward) 32
// registers of column sums, three waves and more fit a SIMD.  One wave per
// row of 512 packs, 8 packs per lane, took 256 registers: 99 us for 16,381 x
// 4096 bf16 rows against 58 us (4.7 TB/s).
struct Shape {
    int lanes, packs;
};

// Rows of more than 2048 packs: forward 4 packs per lane without a row ahead;
// backward the column sums alone would fill the registers, and the two-read
// kernels are faster (4096 x 30000 bf16: 728 us against 579 us).
Shape shape_of(int64_t N, int pack, bool backward) {
    const int64_t packs = (N + pack - 1) / pack;
    if (packs <= 4) return {4, 1};
    if (packs <= 8) return {8, 1};
    if (packs <= 16) return {16, 1};
    if (packs <= 32) return {32, 1};
    if (packs <= 64) return {64, 1};
    if (packs <= 128) return {64, 2};
    if (packs <= 256) return {128, 2};
    if (packs <= 512) return {256, 2};
    if (packs <= 1024) return {512, 2};
    if (packs <= 2048) return {1024, 2};
    if (packs <= 4096 && !backward) return {1024, 4};
    return {0, 0};
}

int pack_of(int type) { return type == SPMM_F32 ? 4 : 8; }

// Blocks that walk the rows: at most `waves` waves on each of 256 compute
// units, so that the weights are loaded and the partial sums written rarely.
int64_t walk_blocks(int64_t R, const Shape &s, int64_t waves) {
    const int block = std::max(256, s.lanes), rows = block / s.lanes;
    const int64_t want = (R + rows - 1) / rows, most = 256 * std::max<int64_t>(1, waves * kWave / block);
    return std::max<int64_t>(1, std::min(want, most));
}

// Forward: 32 waves, 16 where a wave takes several rows (1,000,000 x 64 fp32:
// 88 us against 103 us; 200,000 x 100 bf16: 23 against 22 us).
int64_t forward_blocks(int64_t R, const Shape &s) { return walk_blocks(R, s, s.lanes < kWave ? 16 : 32); }

// Backward: each wave keeps two rows and their sums in flight, and the
// partial sums cost 16 N bytes for each block that writes them: 8 waves, 12
// where a wave takes several rows (65,536 x 1024 bf16: 79 us against 85 us
// with 12 and 90 us with 24; 1,000,000 x 64 fp32: 149, 140 and 161 us).
int64_t backward_blocks(int64_t R, int64_t N, int type) {
    const Shape s = shape_of(N, pack_of(type), true);
    return walk_blocks(R, s, s.lanes < kWave ? 12 : 8);
}

constexpr int64_t kLongBlocks = 2048;

int64_t long_chunks(int64_t R) { return std::max<int64_t>(1, std::min<int64_t>(64, (R + 63) / 64)); }

template <typename T, typename W>
hipError_t norm(const NormArgs &a, hipStream_t s) {
    const Shape sh = shape_of(a.N, kPack<T>, false);
    if (a.R == 0) return hipSuccess;
    if (sh.lanes == 0) {
        norm_long_kernel<T><<<(unsigned)std::min<int64_t>(a.R, kLongBlocks), kLongLanes, 0, s>>>(a);
        return hipGetLastError();
    }
    const unsigned blocks = (unsigned)forward_blocks(a.R, sh);
    const bool stream = 2 * a.R * a.N * (int64_t)sizeof(T) > kStreamBytes;
    const int key = a.N < kPack<T> ? 0 : sh.lanes * 16 + sh.packs;
#define NORM_CASE(G, NV) \
    case G * 16 + NV: norm_kernel<T, W, G, NV><<<blocks, kBlockOf<G>, 0, s>>>(a, stream); break;
    switch (key) {
        NORM_CASE(4, 1) NORM_CASE(8, 1) NORM_CASE(16, 1) NORM_CASE(32, 1) NORM_CASE(64, 1) NORM_CASE(64, 2)
        NORM_CASE(128, 2) NORM_CASE(256, 2) NORM_CASE(512, 2) NORM_CASE(1024, 2)
        case 0: norm_kernel<T, W, 4, 1, true><<<blocks, 256, 0, s>>>(a, stream); break;
        default: norm_kernel<T, W, 1024, 4><<<blocks, 1024, 0, s>>>(a, stream);
    }
#undef NORM_CASE
    return hipGetLastError();
}

template <typename T, typename W>
hipError_t norm_backward(const NormArgs &a, int type, hipStream_t s) {
    const Shape sh = shape_of(a.N, kPack<T>, true);
    NormArgs b = a;
    const bool sums = a.dweight || a.dbias;
    if (!sums) b.partial = nullptr;
    int64_t parts;
    if (sh.lanes == 0) {
        if (a.dx && a.R > 0) {
            norm_backward_long_kernel<T><<<(unsigned)std::min<int64_t>(a.R, kLongBlocks), kLongLanes, 0, s>>>(b);
            if (const hipError_t e = hipGetLastError()) return e;
        }
        parts = long_chunks(a.R);
        if (sums) {
            const int64_t cols = (a.N + 256 * kPack<T> - 1) / (256 * kPack<T>);
            norm_columns_kernel<T><<<dim3((unsigned)cols, (unsigned)parts), 256, 0, s>>>(b, (a.R + parts - 1) / parts);
        }
    } else {
        parts = backward_blocks(a.R, a.N, type);
        const unsigned blocks = (unsigned)parts;
        const bool stream = 3 * a.R * a.N * (int64_t)sizeof(T) > kStreamBytes;
        const int key = a.N < kPack<T> ? 0 : sh.lanes * 16 + sh.packs;
#define NORM_CASE(G, NV) \
    case G * 16 + NV: norm_backward_kernel<T, W, G, NV><<<blocks, kBlockOf<G>, 0, s>>>(b, stream); break;
        switch (key) {
            NORM_CASE(4, 1) NORM_CASE(8, 1) NORM_CASE(16, 1) NORM_CASE(32, 1) NORM_CASE(64, 1) NORM_CASE(64, 2)
            NORM_CASE(128, 2) NORM_CASE(256, 2) NORM_CASE(512, 2)
            case 0: norm_backward_kernel<T, W, 4, 1, true><<<blocks, 256, 0, s>>>(b, stream); break;
            default: norm_backward_kernel<T, W, 1024, 2><<<blocks, 1024, 0, s>>>(b, stream);
        }
#undef NORM_CASE
    }
    if (const hipError_t e = hipGetLastError()) return e;
    if (sums)
        norm_fold_kernel<T><<<(unsigned)((2 * a.N + kFoldColumns - 1) / kFoldColumns), kFoldColumns * kFoldParts, 0,
                              s>>>(b, parts);
    return hipGetLastError();
}

}  // namespace

int64_t norm_workspace_floats(int64_t R, int64_t N, int type) {
    return 2 * N * (shape_of(N, pack_of(type), true).lanes ? backward_blocks(R, N, type) : long_chunks(R));
}

hipError_t launch_norm(const NormArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return norm<float, float>(a, s);
    if (type == SPMM_BF16) return a.weight_fp32 ? norm<__bf16, float>(a, s) : norm<__bf16, __bf16>(a, s);
    return a.weight_fp32 ? norm<_Float16, float>(a, s) : norm<_Float16, _Float16>(a, s);
}

hipError_t launch_norm_backward(const NormArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return norm_backward<float, float>(a, type, s);
    if (type == SPMM_BF16)
        return a.weight_fp32 ? norm_backward<__bf16, float>(a, type, s) : norm_backward<__bf16, __bf16>(a, type, s);
    return a.weight_fp32 ? norm_backward<_Float16, float>(a, type, s) : norm_backward<_Float16, _Float16>(a, type, s);
}

}  // namespace gspmm
