// Dropout: y[i] = residual[i] + (kept(i) ? x[i] / (1 - p) : 0), and with dy in
// place of x and no residual its own gradient.
//
// kept(i) is a function of the element's number alone, so no mask is stored:
// element i takes word i % 4 of the 128 random bits that Philox 4x32 with 10
// rounds (Salmon et al. 2011) makes of the counter (i / 4, offset) and the key
// `seed`, and is kept where that word is at least p * 2^32.  Types, widths and
// launches do not enter, so the mask of a call can be made again anywhere.
//
// Bound by memory: 8 bytes an fp32 element, 4 (6 with a residual) a 16-bit one.
// The generator is 20 products of 32 x 32 bits for four elements.  1,000,000 x 64 fp32,
// forward and backward 83 us each (6.1 TB/s), 16,381 x 4096 bf16 67 us with a residual
// (6.0) and 50 without (5.4).
#include "rows.h"

#include <algorithm>

namespace gspmm {

namespace {

constexpr int kThreads = 256;

struct Words {
    uint32_t w[4];
};

__device__ inline Words random_words(uint64_t group, uint64_t offset, uint64_t key) {
    uint32_t a = (uint32_t)group, b = (uint32_t)(group >> 32), c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t first = (uint64_t)a * 0xD2511F53u, second = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(second >> 32) ^ b ^ k0;
        b = (uint32_t)second;
        c = (uint32_t)(first >> 32) ^ d ^ k1;
        d = (uint32_t)first;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {{a, b, c, d}};
}

// A lane takes packs of 16 bytes.  A dropped element's x is not looked at, so
// what stands there (NaN, infinities) reaches nothing.
template <typename T, bool RESIDUAL>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a, int64_t packs, bool stream) {
    const uint64_t key = (uint64_t)*a.seed;
    const T *x = (const T *)a.x, *res = (const T *)a.residual;
    T *y = (T *)a.y;
    for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < packs; p += (int64_t)gridDim.x * kThreads) {
        const int64_t i = p * kPack<T>, n = a.n - i;
        const Pack<T> in = stream ? load_pack_stream(x + i, n) : load_pack(x + i, n);
        Pack<T> add, out;
        if constexpr (RESIDUAL) add = stream ? load_pack_stream(res + i, n) : load_pack(res + i, n);
#pragma unroll
        for (int g = 0; g < kPack<T> / 4; ++g) {
            const Words r = random_words((uint64_t)(i / 4 + g), (uint64_t)a.offset, key);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool kept = r.w[e] >= a.below && !a.none;
                const float v = (float)in.v[g * 4 + e];
                if constexpr (RESIDUAL) {
                    const float t = (float)add.v[g * 4 + e];
                    out.v[g * 4 + e] = (T)(kept ? fmaf(v, a.scale, t) : t);
                } else {
                    out.v[g * 4 + e] = (T)(kept ? v * a.scale : 0.0f);
                }
            }
        }
        if (stream) store_pack_stream(y + i, out, n);
        else store_pack(y + i, out, n);
    }
}

// Non-temporal accesses where a call moves more than half of the 256 MB
// Infinity Cache: what it reads and writes is then not found there anyway.
constexpr int64_t kStreamBytes = int64_t(128) << 20;
constexpr int64_t kMaxBlocks = 256 * 32;

template <typename T>
hipError_t dropout(const DropoutArgs &a, hipStream_t s) {
    if (a.n == 0) return hipSuccess;
    const int64_t packs = (a.n + kPack<T> - 1) / kPack<T>;
    const unsigned blocks = (unsigned)std::min((packs + kThreads - 1) / kThreads, kMaxBlocks);
    const bool stream = a.n * (int64_t)sizeof(T) * (a.residual ? 3 : 2) > kStreamBytes;
    if (a.residual) dropout_kernel<T, true><<<blocks, kThreads, 0, s>>>(a, packs, stream);
    else dropout_kernel<T, false><<<blocks, kThreads, 0, s>>>(a, packs, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs &a, int type, hipStream_t s) {
    if (type == SPMM_F32) return dropout<float>(a, s);
    if (type == SPMM_BF16) return dropout<__bf16>(a, s);
    return dropout<_Float16>(a, s);
}

}  // namespace gspmm
