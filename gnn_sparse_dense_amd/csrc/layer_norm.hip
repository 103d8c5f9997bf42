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
// is what bounds both.  A group keeps its columns while it walks rows, so the
// weights stay in registers and the backward pass adds dy * u and dy of its
// columns in fp32 registers; at its end a block adds its groups' sums and
// writes one partial row per gradient, and a second kernel adds the partial
// rows in block order (no atomics).  Rows longer than 1024 lanes x 4 packs
// are read from memory once per sum instead.
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kWave = 64;


// Sums of NS values over the group of G lanes, in every lane.  Groups of more
// than a wave are the block; sh holds NS floats per wave, and the caller
// alternates between two of them so that one barrier is enough.
template <int G, int NS>
__device__ inline void group_sum(float (&v)[NS], float *sh) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int o = (G < kWave ? G : kWave) / 2; o > 0; o >>= 1) v[i] += __shfl_xor(v[i], o, kWave);
    }
    if constexpr (G > kWave) {
        constexpr int kWaves = G / kWave;
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) sh[wave * NS + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) t += sh[w * NS + i];
            v[i] = t;
        }
    }
}

template <int G>
constexpr int kBlockOf = G > 256 ? G : 256;

template <typename T, int G, int NV>
__global__ __launch_bounds__(kBlockOf<G>) void norm_kernel(NormArgs a) {
    constexpr int P = kPack<T>, kRows = kBlockOf<G> / G;
    __shared__ float sh[2][G > kWave ? G / kWave : 1];
    const int lane = threadIdx.x % G;
    const float inv_n = 1.0f / (float)a.N;
    float weight[NV][P], bias[NV][P];
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t c = ((int64_t)q * G + lane) * P + i;
            weight[q][i] = a.weight && c < a.N ? load_weight<T>(a.weight, c, a.weight_fp32) : 1.0f;
            bias[q][i] = a.bias && c < a.N ? load_weight<T>(a.bias, c, a.weight_fp32) : 0.0f;
        }
    // every group of a block takes the same number of turns (the barriers)
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.R; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t r = r0 + threadIdx.x / G;
        const bool live = r < a.R;
        Pack<T> x[NV];
        float s[1] = {0.0f};
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t c = ((int64_t)q * G + lane) * P;
            x[q] = load_pack((const T *)a.x + r * a.N + c, live ? a.N - c : 0);
#pragma unroll
            for (int i = 0; i < P; ++i) s[0] += (float)x[q].v[i];
        }
        group_sum<G, 1>(s, sh[0]);
        const float mean = s[0] * inv_n;
        s[0] = 0.0f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t c = ((int64_t)q * G + lane) * P + i;
                const float d = (float)x[q].v[i] - mean;
                if (c < a.N) s[0] = fmaf(d, d, s[0]);
            }
        group_sum<G, 1>(s, sh[1]);
        const float rstd = 1.0f / sqrtf(s[0] * inv_n + a.eps);
        if (!live) continue;
        if (lane == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t c = ((int64_t)q * G + lane) * P;
            Pack<T> y;
#pragma unroll
            for (int i = 0; i < P; ++i)
                y.v[i] = (T)fmaf(((float)x[q].v[i] - mean) * rstd, weight[q][i], bias[q][i]);
            store_pack((T *)a.y + r * a.N + c, y, a.N - c);
        }
    }
}

// Rows too long for registers: one block per row, three reads.
template <typename T>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    constexpr int G = 1024, P = kPack<T>;
    __shared__ float sh[2][G / kWave];
    const float inv_n = 1.0f / (float)a.N;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        const T *x = (const T *)a.x + r * a.N;
        float s[1] = {0.0f};
        for (int64_t c = (int64_t)threadIdx.x * P; c < a.N; c += G * P) {
            const Pack<T> v = load_pack(x + c, a.N - c);
#pragma unroll
            for (int i = 0; i < P; ++i) s[0] += (float)v.v[i];
        }
        group_sum<G, 1>(s, sh[0]);
        const float mean = s[0] * inv_n;
        s[0] = 0.0f;
        for (int64_t c = (int64_t)threadIdx.x * P; c < a.N; c += G * P) {
            const Pack<T> v = load_pack(x + c, a.N - c);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float d = (float)v.v[i] - mean;
                if (c + i < a.N) s[0] = fmaf(d, d, s[0]);
            }
        }
        group_sum<G, 1>(s, sh[1]);
        const float rstd = 1.0f / sqrtf(s[0] * inv_n + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        for (int64_t c = (int64_t)threadIdx.x * P; c < a.N; c += G * P) {
            const Pack<T> v = load_pack(x + c, a.N - c);
            Pack<T> y;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const bool in = c + i < a.N;
                const float w = a.weight && in ? load_weight<T>(a.weight, c + i, a.weight_fp32) : 1.0f;
                const float b = a.bias && in ? load_weight<T>(a.bias, c + i, a.weight_fp32) : 0.0f;
                y.v[i] = (T)fmaf(((float)v.v[i] - mean) * rstd, w, b);
            }
            store_pack((T *)a.y + r * a.N + c, y, a.N - c);
        }
    }
}

// partial: [gridDim.x][2][N] (dweight, dbias), written when a.partial is set.
template <typename T, int G, int NV>
__global__ __launch_bounds__(kBlockOf<G>) void norm_backward_kernel(NormArgs a) {
    constexpr int P = kPack<T>, kRows = kBlockOf<G> / G;
    __shared__ float sh[2][G > kWave ? 2 * G / kWave : 1];
    const int lane = threadIdx.x % G;
    const float inv_n = 1.0f / (float)a.N;
    float weight[NV][P], dw[NV][P] = {}, db[NV][P] = {};
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t c = ((int64_t)q * G + lane) * P + i;
            weight[q][i] = a.weight && c < a.N ? load_weight<T>(a.weight, c, a.weight_fp32) : 1.0f;
        }
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.R; r0 += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t r = r0 + threadIdx.x / G;
        const bool live = r < a.R;
        const float mean = live ? a.mean[r] : 0.0f, rstd = live ? a.rstd[r] : 0.0f;
        Pack<T> x[NV], d[NV];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t c = ((int64_t)q * G + lane) * P, n = live ? a.N - c : 0;
            x[q] = load_pack((const T *)a.x + r * a.N + c, n);
            d[q] = load_pack((const T *)a.dy + r * a.N + c, n);
        }
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t c = ((int64_t)q * G + lane) * P + i;
                const float u = live && c < a.N ? ((float)x[q].v[i] - mean) * rstd : 0.0f;
                const float dy = (float)d[q].v[i], g = dy * weight[q][i];
                s[0] += g;
                s[1] = fmaf(g, u, s[1]);
                dw[q][i] = fmaf(dy, u, dw[q][i]);
                db[q][i] += dy;
            }
        if (!a.dx) continue;                        // the same for every lane
        group_sum<G, 2>(s, sh[turn]);
        const float mg = s[0] * inv_n, mgu = s[1] * inv_n;
        if (!live) continue;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int64_t c = ((int64_t)q * G + lane) * P;
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float u = ((float)x[q].v[i] - mean) * rstd, g = (float)d[q].v[i] * weight[q][i];
                o.v[i] = (T)(rstd * (g - mg - u * mgu));
            }
            store_pack((T *)a.dx + r * a.N + c, o, a.N - c);
        }
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
    if constexpr (G <= kWave) {
        constexpr int kWaves = kBlockOf<G> / kWave, kLanes = G < kWave ? G : kWave;
        __shared__ float acc[kWaves][2][NV][P][kLanes];
        const int wave = threadIdx.x / kWave, at = threadIdx.x % kWave;
        if (at < kLanes)
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    acc[wave][0][q][i][at] = dw[q][i];
                    acc[wave][1][q][i][at] = db[q][i];
                }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * NV * P * kLanes; i += kBlockOf<G>) {
            const int l = i % kLanes, e = i / kLanes % P, q = i / (kLanes * P) % NV, which = i / (kLanes * P * NV);
            const int64_t c = ((int64_t)q * G + l) * P + e;
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) t += acc[w][which][q][e][l];
            if (c < a.N) out[which * a.N + c] = t;
        }
    } else {
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t c = ((int64_t)q * G + lane) * P + i;
                if (c < a.N) {
                    out[c] = dw[q][i];
                    out[a.N + c] = db[q][i];
                }
            }
    }
}

// Rows too long for registers: dx with two reads of the row.
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(NormArgs a) {
    constexpr int G = 1024, P = kPack<T>;
    __shared__ float sh[2][2 * G / kWave];
    const float inv_n = 1.0f / (float)a.N;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        const T *x = (const T *)a.x + r * a.N, *dy = (const T *)a.dy + r * a.N;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = (int64_t)threadIdx.x * P; c < a.N; c += G * P) {
            const Pack<T> v = load_pack(x + c, a.N - c), d = load_pack(dy + c, a.N - c);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float w = a.weight && c + i < a.N ? load_weight<T>(a.weight, c + i, a.weight_fp32) : 1.0f;
                const float u = c + i < a.N ? ((float)v.v[i] - mean) * rstd : 0.0f, g = (float)d.v[i] * w;
                s[0] += g;
                s[1] = fmaf(g, u, s[1]);
            }
        }
        group_sum<G, 2>(s, sh[turn]);
        const float mg = s[0] * inv_n, mgu = s[1] * inv_n;
        for (int64_t c = (int64_t)threadIdx.x * P; c < a.N; c += G * P) {
            const Pack<T> v = load_pack(x + c, a.N - c), d = load_pack(dy + c, a.N - c);
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float w = a.weight && c + i < a.N ? load_weight<T>(a.weight, c + i, a.weight_fp32) : 1.0f;
                const float u = ((float)v.v[i] - mean) * rstd, g = (float)d.v[i] * w;
                o.v[i] = (T)(rstd * (g - mg - u * mgu));
            }
            store_pack((T *)a.dx + r * a.N + c, o, a.N - c);
        }
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

// dweight / dbias: partial rows added in order, each thread a strided part of
// them, the parts added in order.  64 columns of one gradient per block.
constexpr int kFoldParts = 16;

template <typename T>
__global__ __launch_bounds__(kWave *kFoldParts) void norm_fold_kernel(NormArgs a, int64_t parts) {
    __shared__ float sh[kFoldParts][kWave];
    const int lane = threadIdx.x % kWave, part = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWave + lane;      // over [2][N]
    float t = 0.0f;
    if (c < 2 * a.N)
        for (int64_t p = part; p < parts; p += kFoldParts) t += a.partial[p * 2 * a.N + c];
    sh[part][lane] = t;
    __syncthreads();
    if (part != 0 || c >= 2 * a.N) return;
#pragma unroll
    for (int p = 1; p < kFoldParts; ++p) t += sh[p][lane];
    void *out = c < a.N ? a.dweight : a.dbias;
    if (out) store_weight<T>(out, c < a.N ? c : c - a.N, a.weight_fp32, t);
}

// ---- shapes ----

// Lanes of a row's group and packs per lane; 0 lanes: too long for registers.
struct Shape {
    int lanes, packs;
};

Shape shape_of(int64_t N, int pack) {
    const int64_t packs = (N + pack - 1) / pack;
    if (packs <= 4) return {4, 1};
    if (packs <= 8) return {8, 1};
    if (packs <= 16) return {16, 1};
    if (packs <= 32) return {32, 1};
    if (packs <= 64) return {64, 1};
    if (packs <= 128) return {64, 2};
    if (packs <= 256) return {256, 1};
    if (packs <= 512) return {256, 2};
    if (packs <= 1024) return {1024, 1};
    if (packs <= 2048) return {1024, 2};
    if (packs <= 4096) return {1024, 4};
    return {0, 0};
}

int pack_of(int type) { return type == SPMM_F32 ? 4 : 8; }

// Blocks that walk the rows: enough waves to fill 256 compute units, few
// enough that the weights are loaded and the partial sums written rarely.
int64_t walk_blocks(int64_t R, const Shape &s) {
    const int block = std::max(256, s.lanes), rows = block / s.lanes;
    const int64_t want = (R + rows - 1) / rows, most = 256 * (2048 / block);
    return std::max<int64_t>(1, std::min(want, most));
}

constexpr int64_t kLongBlocks = 2048;

int64_t long_chunks(int64_t R) { return std::max<int64_t>(1, std::min<int64_t>(64, (R + 63) / 64)); }

template <typename T>
hipError_t norm(const NormArgs &a, hipStream_t s) {
    const Shape sh = shape_of(a.N, kPack<T>);
    if (a.R == 0) return hipSuccess;
    if (sh.lanes == 0) {
        norm_long_kernel<T><<<(unsigned)std::min<int64_t>(a.R, kLongBlocks), 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    const unsigned blocks = (unsigned)walk_blocks(a.R, sh);
    const int key = sh.lanes * 8 + sh.packs;
#define NORM_CASE(G, NV) \
    case G * 8 + NV: norm_kernel<T, G, NV><<<blocks, kBlockOf<G>, 0, s>>>(a); break;
    switch (key) {
        NORM_CASE(4, 1) NORM_CASE(8, 1) NORM_CASE(16, 1) NORM_CASE(32, 1) NORM_CASE(64, 1) NORM_CASE(64, 2)
        NORM_CASE(256, 1) NORM_CASE(256, 2) NORM_CASE(1024, 1) NORM_CASE(1024, 2) NORM_CASE(1024, 4)
        default: return hipErrorInvalidValue;
    }
#undef NORM_CASE
    return hipGetLastError();
}

template <typename T>
hipError_t norm_backward(const NormArgs &a, hipStream_t s) {
    const Shape sh = shape_of(a.N, kPack<T>);
    NormArgs b = a;
    const bool sums = a.dweight || a.dbias;
    if (!sums) b.partial = nullptr;
    int64_t parts;
    if (sh.lanes == 0) {
        if (a.dx && a.R > 0) {
            norm_backward_long_kernel<T><<<(unsigned)std::min<int64_t>(a.R, kLongBlocks), 1024, 0, s>>>(b);
            if (const hipError_t e = hipGetLastError()) return e;
        }
        parts = long_chunks(a.R);
        if (sums) {
            const int64_t cols = (a.N + 256 * kPack<T> - 1) / (256 * kPack<T>);
            norm_columns_kernel<T><<<dim3((unsigned)cols, (unsigned)parts), 256, 0, s>>>(b, (a.R + parts - 1) / parts);
        }
    } else {
        parts = walk_blocks(a.R, sh);
        const unsigned blocks = (unsigned)parts;
        const int key = sh.lanes * 8 + sh.packs;
#define NORM_CASE(G, NV) \
    case G * 8 + NV: norm_backward_kernel<T, G, NV><<<blocks, kBlockOf<G>, 0, s>>>(b); break;
        switch (key) {
            NORM_CASE(4, 1) NORM_CASE(8, 1) NORM_CASE(16, 1) NORM_CASE(32, 1) NORM_CASE(64, 1) NORM_CASE(64, 2)
            NORM_CASE(256, 1) NORM_CASE(256, 2) NORM_CASE(1024, 1) NORM_CASE(1024, 2) NORM_CASE(1024, 4)
            default: return hipErrorInvalidValue;
        }
#undef NORM_CASE
    }
    if (const hipError_t e = hipGetLastError()) return e;
    if (sums) norm_fold_kernel<T><<<(unsigned)((2 * a.N + kWave - 1) / kWave), kWave * kFoldParts, 0, s>>>(b, parts);
    return hipGetLastError();
}

}  // namespace

int64_t norm_workspace_floats(int64_t R, int64_t N, int type) {
    const Shape sh = shape_of(N, pack_of(type));
    return 2 * N * (sh.lanes ? walk_blocks(R, sh) : long_chunks(R));
}

hipError_t launch_norm(const NormArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return norm<float>(a, s);
    if (type == SPMM_BF16) return norm<__bf16>(a, s);
    return norm<_Float16>(a, s);
}

hipError_t launch_norm_backward(const NormArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return norm_backward<float>(a, s);
    if (type == SPMM_BF16) return norm_backward<__bf16>(a, s);
    return norm_backward<_Float16>(a, s);
}

}  // namespace gspmm
