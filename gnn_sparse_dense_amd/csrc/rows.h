// Device-side helpers and argument structs of the row operators: the routed
// exchange (rows sorted by expert and back), the segment product and the
// layer norm.  Rows are packed row-major in fp32, bf16 or fp16; arithmetic is
// fp32 throughout and every output is rounded once, when it is stored.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "spmm.h"

namespace gspmm {

// 16 bytes of a row.  Loads and stores go through memcpy from an
// element-aligned address: gfx950 takes global_load/store_dwordx4 at any
// element alignment, so odd widths keep the wide accesses.
template <typename T>
constexpr int kPack = 16 / (int)sizeof(T);

template <typename T>
struct alignas(16) Pack {
    T v[16 / sizeof(T)];
};

template <typename T>
__device__ inline Pack<T> load_pack(const T *p) {
    Pack<T> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}

// The first n elements (n <= 0: none); the others are zero.
template <typename T>
__device__ inline Pack<T> load_pack(const T *p, int64_t n) {
    if (n >= kPack<T>) return load_pack(p);
    Pack<T> r;
#pragma unroll
    for (int i = 0; i < kPack<T>; ++i) r.v[i] = i < n ? p[i] : (T)0.0f;
    return r;
}

template <typename T>
__device__ inline void store_pack(T *p, const Pack<T> &r, int64_t n) {
    if (n >= kPack<T>) {
        __builtin_memcpy(p, &r, sizeof(r));
        return;
    }
#pragma unroll
    for (int i = 0; i < kPack<T>; ++i)
        if (i < n) p[i] = r.v[i];
}

// Streaming accesses: non-temporal, so that what is written once (or read
// once) does not displace what is read again from the 256 MB Infinity Cache.
template <int ALIGN>
struct Stream;
template <>
struct Stream<2> {
    typedef int V __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Stream<4> {
    typedef int V __attribute__((ext_vector_type(4), aligned(4)));
};

template <typename T>
__device__ inline Pack<T> load_pack_stream(const T *p, int64_t n) {
    typedef typename Stream<sizeof(T)>::V V;
    if (n >= kPack<T>) return __builtin_bit_cast(Pack<T>, __builtin_nontemporal_load((const V *)p));
    return load_pack(p, n);
}

template <typename T>
__device__ inline void store_pack_stream(T *p, const Pack<T> &r, int64_t n) {
    typedef typename Stream<sizeof(T)>::V V;
    if (n >= kPack<T>) __builtin_nontemporal_store(__builtin_bit_cast(V, r), (V *)p);
    else store_pack(p, r, n);
}

// A weight stored in fp32 or in the rows' own type.
template <typename T>
__device__ inline float load_weight(const void *w, int64_t i, bool fp32) {
    return fp32 ? static_cast<const float *>(w)[i] : (float)static_cast<const T *>(w)[i];
}

template <typename T>
__device__ inline void store_weight(void *w, int64_t i, bool fp32, float v) {
    if (fp32) static_cast<float *>(w)[i] = v;
    else static_cast<T *>(w)[i] = (T)v;
}

// ---- the route and the exchange (exchange.hip) ----

constexpr int kRouteMaxExperts = 2048;

struct RouteArgs {
    const int64_t *expert;   // [pairs]; values outside [0, E): no expert
    int64_t pairs;
    int E;
    int64_t *offsets;        // [E + 1]
    int *order;              // [pairs]
    int *position;           // [pairs]
    int *workspace;          // route_workspace_ints(pairs, E)
};
int64_t route_workspace_ints(int64_t pairs, int64_t E);
hipError_t launch_route(const RouteArgs &a, hipStream_t s);

struct ExchangeArgs {
    const int64_t *offsets;  // [E + 1]; rows from offsets[E] on belong to no expert
    const int *position;     // [T, k] (combine)
    const int *order;        // [T * k] (dispatch, combine's gradients)
    int64_t T;
    int64_t k;
    int64_t E;
    int64_t N;
    const void *rows;        // dispatch: [T, N]; combine: [T * k, N]
    const void *weight;      // [T, k] or nullptr (1)
    int weight_fp32;
    void *out;               // dispatch: [T * k, N]; combine: [T, N]
    const void *dout;        // combine's gradients: [T, N]
    void *drows;             // [T * k, N] or nullptr
    void *dweight;           // [T, k]
};
hipError_t launch_dispatch(const ExchangeArgs &a, int type, hipStream_t s);
hipError_t launch_combine(const ExchangeArgs &a, int type, hipStream_t s);
hipError_t launch_combine_backward(const ExchangeArgs &a, int type, hipStream_t s);

// ---- the layer norm (layer_norm.hip) ----

struct NormArgs {
    const void *x;           // [R, N]
    const void *weight;      // [N] or nullptr (1)
    const void *bias;        // [N] or nullptr (0)
    int weight_fp32;
    float eps;
    int64_t R;
    int64_t N;
    void *y;                 // [R, N]
    float *mean;             // [R] or nullptr
    float *rstd;             // [R] or nullptr
    const void *dy;          // [R, N]
    void *dx;                // [R, N] or nullptr
    void *dweight;           // [N] or nullptr
    void *dbias;             // [N] or nullptr
    float *partial;          // norm_workspace_floats(R, N)
};
int64_t norm_workspace_floats(int64_t R, int64_t N, int type);
hipError_t launch_norm(const NormArgs &a, int type, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, int type, hipStream_t s);

// ---- the segment product (segment.hip) ----

struct SegmentArgs {
    const int64_t *offsets;  // [E + 1]
    int64_t R;               // rows of a
    int64_t E;
    int64_t I;               // w is [E, I, O]
    int64_t O;
    const void *x;           // [R, I]
    const void *w;           // [E, I, O]
    const void *dy;          // [R, O]
    void *y;                 // product: [R, O]; transposed: [R, I]; dw: [E, I, O]
    float *partial;          // dw: segment_workspace_floats(...)
};
int64_t segment_workspace_floats(int64_t R, int64_t E, int64_t I, int64_t O, int type);
hipError_t launch_segment(const SegmentArgs &a, bool transposed, int type, hipStream_t s);
hipError_t launch_segment_dw(const SegmentArgs &a, int type, hipStream_t s);

}  // namespace gspmm
