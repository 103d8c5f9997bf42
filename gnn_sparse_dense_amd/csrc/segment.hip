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
// A block computes one tile of the output (tile_product.h).
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
#include "tile_product.h"

namespace gspmm {

namespace {

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
    TILE_STAGES(lds, S::kStageBytes);
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
    TILE_STAGES(lds, S::kStageBytes);
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
