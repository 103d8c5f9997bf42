"""The segment product's 16-bit kernels for large calls, every output against
64 bits: 256 x 256 tiles of y, dx and dw, and dw in chunks of rows.
Tolerances as for the small calls: a product's terms count 2 u each, and an
output is rounded once."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24

# E, I, O: 512 tiles of 256 x 256 and more; 1 to 72 tiles to a segment, at most and above 64 segments
DW_LARGE = [(32, 1000, 1032), (32, 1024, 1024), (70, 520, 776), (130, 264, 520), (9, 1800, 2056), (520, 64, 48),
            (64, 512, 1040), (65, 1016, 512)]
# R, E, I, O: more than 4,096 rows and fewer tiles; whole 16-byte groups and not
DW_CHUNKS = [(20011, 5, 264, 136), (20011, 5, 265, 131), (20011, 5, 1024, 1024), (4097, 1, 8, 8), (40000, 70, 72, 16),
             (30000, 3, 1, 3), (9000, 40, 129, 250)]
# R, E, I, O: 512 tiles of y or of dx and more, ragged in rows and columns; the
# summed index in whole rounds of four 64-byte steps and not
PRODUCT = [(16500, 40, 328, 2056), (16500, 40, 2056, 328), (16400, 300, 264, 2048), (16400, 300, 2048, 264),
           (19000, 7, 1544, 1544), (131080, 33, 8, 24), (131080, 5, 296, 256), (131080, 5, 256, 296)]


def close(got, ref, before, dtype, what):
    err = (got.double() - ref).abs()
    f = torch.finfo(dtype)
    size = ref.abs() + before
    bad = ~(err <= 1.01 * (before + size * (f.eps / 2) + f.smallest_normal * f.eps / 2))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error {float(err.max()):.3e}"


def inputs(R, bounds, E, I, O, dtype, seed):
    """Rows outside the segments hold NaN and infinities."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x, w, dy = (torch.randn(*s, generator=g, device=DEV).to(dtype) for s in ((R, I), (E, I, O), (R, O)))
    for a, b in ((0, bounds[0]), (bounds[-1], R)):
        x[a:b] = float("nan")
        dy[a:b] = float("inf")
    return x, w, dy, torch.tensor(bounds, device=DEV)


def uneven(R, E, head, tail, seed):
    """Bounds of E segments of random lengths, some in the middle empty."""
    g = torch.Generator()
    g.manual_seed(seed)
    cut = torch.sort(torch.randint(head, R - tail + 1, (E - 1,), generator=g)).values.tolist()
    cut[E // 3:E // 2] = cut[E // 3:E // 3 + 1] * len(cut[E // 3:E // 2])
    return [head, *cut, R - tail]


def check_dw(dw, x, dy, bounds, dtype):
    for e in range(len(bounds) - 1):
        X, D = (t[bounds[e]:bounds[e + 1]].double() for t in (x, dy))
        Xt = X.t().contiguous()
        close(dw[e], Xt @ D, 2 * U * max(1, X.shape[0]) * (Xt.abs() @ D.abs()), dtype, f"dw of segment {e}")


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("E,I,O", DW_LARGE)
def test_dw_of_large_tiles(E, I, O, kind):
    """Segments of no row, of one, and around whole 32-row steps and rounds of four."""
    log(f"dw large E={E} I={I} O={O} {kind}")
    lengths = [0, 1, 31, 32, 33, 64, 97, 127, 128, 129, 0, 160, 255, 300, 2]
    bounds = [3]
    for e in range(E):
        bounds.append(bounds[-1] + lengths[e % len(lengths)])
    x, w, dy, b = inputs(bounds[-1] + 130, bounds, E, I, O, TYPES[kind], E + I)
    dw = torch.full_like(w, float("nan"))
    G.spmm_segment_product_dw(x, dy, b, dw)
    check_dw(dw, x, dy, bounds, TYPES[kind])


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,E,I,O", DW_CHUNKS)
def test_dw_in_chunks_of_rows(R, E, I, O, kind):
    log(f"dw chunks R={R} E={E} I={I} O={O} {kind}")
    bounds = uneven(R, E, 5, 70, R + E)
    x, w, dy, b = inputs(R, bounds, E, I, O, TYPES[kind], R + I)
    dw = torch.full_like(w, float("nan"))
    G.spmm_segment_product_dw(x, dy, b, dw)
    check_dw(dw, x, dy, bounds, TYPES[kind])


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,E,I,O", PRODUCT)
def test_products_of_large_tiles(R, E, I, O, kind):
    log(f"products R={R} E={E} I={I} O={O} {kind}")
    bounds = uneven(R, E, 9, 300, R + E + I)
    dtype = TYPES[kind]
    x, w, dy, b = inputs(R, bounds, E, I, O, dtype, R + I)
    y, dx = torch.full_like(dy, float("nan")), torch.full_like(x, float("nan"))
    G.spmm_segment_product(x, w, b, y)
    G.spmm_segment_product_dx(dy, w, b, dx)
    for e in range(E):
        s = slice(bounds[e], bounds[e + 1])
        X, W, D = x[s].double(), w[e].double(), dy[s].double()
        Wt = W.t().contiguous()
        close(y[s], X @ W, 2 * U * I * (X.abs() @ W.abs()), dtype, f"y of segment {e}")
        close(dx[s], D @ Wt, 2 * U * O * (D.abs() @ Wt.abs()), dtype, f"dx of segment {e}")
    for out in (y, dx):
        assert not bool(out[:bounds[0]].any()) and not bool(out[bounds[-1]:].any())
