// Attention within segments: what a call's shape decides on the host.  The
// kernels and their mathematics are in attention_impl.h.
#include "rows.h"

#include <algorithm>

namespace gspmm {

template <typename T>
hipError_t launch_attention_pass(const AttentionArgs &a, AttentionPass pass, bool large, bool direct, hipStream_t s);
template <typename T>
hipError_t launch_attention_join(const AttentionArgs &a, hipStream_t s);
template <typename T>
hipError_t launch_attention_add(const AttentionArgs &a, bool large, hipStream_t s);

namespace {

// Exact quotients of n < 2^31: (n * magic) >> shift with magic = floor(2^shift / d) + 1.
Divisor divisor(int64_t d) {
    int s = 0;
    while ((int64_t(1) << s) < d) ++s;
    return {(uint32_t)((uint64_t(1) << (31 + s)) / (uint64_t)d + 1), 31 + s, (int)d};
}

// The copy into LDS needs rows of whole 16-byte groups, from a 16-byte address,
// and 32-bit offsets within a tile's rows.
bool direct_rows(const void *p, int64_t ld, int64_t D, int size) {
    return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0 && D * size % 16 == 0 && ld * size < (int64_t(1) << 24);
}

// Tiles of 128 rows by four waves that share their keys, or of 32 by one: by the
// mean length of a segment, since the device alone knows each.  With gradients, 8
// heads, four waves and one: bf16, 64 elements, 256 segments of 64 rows 111 and 92 us,
// 128 of 128 117 and 102, of 256 216 and 222; 128 elements 227 and 174, 244 and 205, 506
// and 575; fp32, 32 elements 159 and 121, 208 and 171, 512 and 452.
bool large_tiles(int64_t rows, int64_t S, int size) { return rows > (size == 4 ? 256 : 128) * S; }

// Parts of a segment's keys that are worked on side by side and joined afterwards,
// where there are too few tiles to fill the chip: about `want` blocks, at least
// `least` keys to a part of a segment of mean length.  One row each, 32 heads of 128
// over 8, bf16: 4 segments of 8,000 keys, 256 to a part 37 us, 128 43, 512 39; 32 of
// 1,000 33, 37 and 47; one of 65,536, at most 64 parts 59 us, 128 66, 256 88.  128-row
// tiles: 3,001 rows to 5,003 keys in 9, 256 keys to a part 30 us, 512 (one part) 27.
int64_t parts_of(int64_t blocks, int64_t want, int64_t keys, int64_t S, int64_t least) {
    const int64_t length = keys / std::max<int64_t>(1, S);
    return std::max<int64_t>(1, std::min({want / std::max<int64_t>(1, blocks), length / least, int64_t(64)}));
}

int query_rows(int64_t R, int64_t S, int64_t H, int64_t Hk, int size) {
    return large_tiles(R * (H / Hk), S, size) ? 128 : 32;
}

int64_t tiles(int64_t rows, int64_t S, bool large) { return rows / (large ? 128 : 32) + std::min(rows, S); }

int query_parts(int64_t R, int64_t K, int64_t S, int64_t H, int64_t Hk, int size) {
    const bool large = large_tiles(R * (H / Hk), S, size);
    return (int)parts_of(tiles(R * (H / Hk), S, large) * Hk, large ? 512 : 2048, K, S, large ? 512 : 256);
}

// Packed rows of a part of a key tile's rows: a third of what a compute unit has to
// take of all tiles (the mean tile's rows; half of them are seen if causal), and
// the most parts that a tile is cut into.
constexpr int64_t kUnits = 256;
constexpr int kMostParts = 16;

int64_t part_rows(int64_t R, int64_t K, int64_t S, int64_t H, int64_t Hk, int size) {
    const int64_t rows = R * (H / Hk) / std::max<int64_t>(1, S);
    const int64_t share = tiles(K, S, large_tiles(K, S, size)) * Hk * rows / (3 * kUnits);
    return std::max<int64_t>(512, share);
}

int key_parts(int64_t R, int64_t K, int64_t S, int64_t H, int64_t Hk, int size) {
    // the longest segment's rows are taken to be thrice the mean
    const int64_t rows = R * (H / Hk) / std::max<int64_t>(1, S);
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMostParts, 3 * rows / part_rows(R, K, S, H, Hk, size)));
}

}  // namespace

int64_t attention_workspace_floats(int64_t R, int64_t K, int64_t S, int64_t H, int64_t Hk, int64_t D, int type) {
    const int64_t parts = query_parts(R, K, S, H, Hk, type == SPMM_F32 ? 4 : 2);
    return parts > 1 ? parts * R * H * (D + 2) : 0;
}

// delta, and in fp16 lse once more and two floats of each wave of dq's blocks.
static int64_t row_floats(int64_t R, int64_t S, int64_t H, int64_t Hk, int type) {
    if (type != SPMM_F16) return R * H;
    const int64_t rows = query_rows(R, S, H, Hk, 2);
    return 2 * R * H + 2 * (R * (H / Hk) / rows + S + 2) * Hk * (rows / 32);
}

int64_t attention_backward_workspace_floats(int64_t R, int64_t K, int64_t S, int64_t H, int64_t Hk, int64_t D,
                                            int type) {
    const int64_t parts = key_parts(R, K, S, H, Hk, type == SPMM_F32 ? 4 : 2);
    return row_floats(R, S, H, Hk, type) + (parts > 1 ? 2 * parts * K * Hk * D : 0);
}

hipError_t launch_attention(const AttentionArgs &args, float *workspace, int type, hipStream_t s) {
    if (args.R == 0) return hipSuccess;
    AttentionArgs a = args;
    const int size = type == SPMM_F32 ? 4 : 2;
    a.G = divisor(a.H / a.Hk);
    a.parts = query_parts(a.R, a.K, a.S, a.H, a.Hk, size);
    if (a.parts > 1) {
        a.partial = workspace;
        a.partial_top = workspace + a.parts * a.R * a.H * a.D;
        a.partial_sum = a.partial_top + a.parts * a.R * a.H;
    }
    const bool large = large_tiles(a.R * a.G.d, a.S, size);
    a.short_keys = a.K <= 64 * a.S;
    const bool direct = direct_rows(a.k, a.ldk, a.D, size) && direct_rows(a.v, a.ldv, a.D, size);
    const auto pass = AttentionPass::kForward;
    if (const hipError_t e = type == SPMM_F32    ? launch_attention_pass<float>(a, pass, large, direct, s)
                             : type == SPMM_BF16 ? launch_attention_pass<__bf16>(a, pass, large, direct, s)
                                                 : launch_attention_pass<_Float16>(a, pass, large, direct, s))
        return e;
    if (a.parts == 1) return hipSuccess;
    return type == SPMM_F32    ? launch_attention_join<float>(a, s)
           : type == SPMM_BF16 ? launch_attention_join<__bf16>(a, s)
                               : launch_attention_join<_Float16>(a, s);
}

hipError_t launch_attention_backward(const AttentionArgs &args, float *workspace, int type, hipStream_t s) {
    AttentionArgs a = args;
    const int size = type == SPMM_F32 ? 4 : 2;
    a.G = divisor(a.H / a.Hk);
    a.parts = 1;
    a.key_parts = key_parts(a.R, a.K, a.S, a.H, a.Hk, size);
    a.part_rows = part_rows(a.R, a.K, a.S, a.H, a.Hk, size) / (a.causal ? 2 : 1);
    a.query_rows = query_rows(a.R, a.S, a.H, a.Hk, size);
    a.delta = workspace;
    a.held_lse = workspace + a.R * a.H;
    a.sizes = a.held_lse + a.R * a.H;
    a.partial_dk = workspace + row_floats(a.R, a.S, a.H, a.Hk, type);
    a.partial_dv = a.partial_dk + a.key_parts * a.K * a.Hk * a.D;
    auto pass = [&](AttentionPass p, bool large, bool direct) {
        return type == SPMM_F32    ? launch_attention_pass<float>(a, p, large, direct, s)
               : type == SPMM_BF16 ? launch_attention_pass<__bf16>(a, p, large, direct, s)
                                   : launch_attention_pass<_Float16>(a, p, large, direct, s);
    };
    if (a.R > 0) {
        const bool direct = direct_rows(a.k, a.ldk, a.D, size) && direct_rows(a.v, a.ldv, a.D, size);
        if (const hipError_t e = pass(AttentionPass::kQueries, large_tiles(a.R * a.G.d, a.S, size), direct)) return e;
    }
    if (a.K == 0 || (!a.dk && !a.dv)) return hipSuccess;
    const bool direct = direct_rows(a.q, a.ldq, a.D, size) && direct_rows(a.dout, a.H * a.D, a.D, size);
    if (const hipError_t e = pass(AttentionPass::kKeys, large_tiles(a.K, a.S, size), direct)) return e;
    if (a.key_parts == 1) return hipSuccess;
    return type == SPMM_F32    ? launch_attention_add<float>(a, large_tiles(a.K, a.S, size), s)
           : type == SPMM_BF16 ? launch_attention_add<__bf16>(a, large_tiles(a.K, a.S, size), s)
                               : launch_attention_add<_Float16>(a, large_tiles(a.K, a.S, size), s);
}

}  // namespace gspmm
