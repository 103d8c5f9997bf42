"""Segment products of more segments than one wave scans: results against 64
bits, and time that grows with the segments and not with their square."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log
    from tests.test_gpu_rows import guarded
    from tests.test_gpu_segment_paths import U, close

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

# R, E, I, O: a few rows to a segment or many, whole 16-byte groups and not, and 256 x 256 tiles of y
MANY = [(3000, 513, 16, 24), (20000, 1000, 33, 7), (200000, 1100, 8, 40), (9001, 5000, 8, 8), (70000, 70000, 8, 16),
        (140000, 70000, 5, 3), (131072, 2000, 8, 264)]


def many(R, E, I, O, dtype):
    """Segments of random lengths, a third of them empty; NaN in the rows around them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(R + E)
    of = torch.randint(0, E, (R - 350,), generator=g, device=DEV)
    of = torch.where(of % 3 == 1, of - 1, of)
    rows = torch.bincount(of, minlength=E)
    b = torch.cat([torch.full((1,), 150, device=DEV), 150 + rows.cumsum(0)])
    x, w, dy = (torch.randn(*s, generator=g, device=DEV).to(dtype) for s in ((R, I), (E, I, O), (R, O)))
    for t in (x, dy):
        t[:150], t[R - 200:] = float("nan"), float("inf")
    return x, w, dy, b, torch.sort(of).values


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,E,I,O", MANY)
def test_products_of_many_segments(R, E, I, O, kind):
    log(f"many R={R} E={E} I={I} O={O} {kind}")
    dtype = TYPES[kind]
    x, w, dy, b, of = many(R, E, I, O, dtype)
    y, dx, dw = torch.full_like(dy, float("nan")), torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    G.spmm_segment_product(x, w, b, y)
    G.spmm_segment_product_dx(dy, w, b, dx)
    G.spmm_segment_product_dw(x, dy, b, dw)
    inside = slice(150, R - 200)
    for out in (y, dx):
        assert not bool(out[:150].any()) and not bool(out[R - 200:].any())
    X, D = x[inside].double(), dy[inside].double()
    want, size = torch.zeros(2, E, I, O, dtype=torch.float64, device=DEV)
    for at in range(0, R - 350, 1 << 14):                # products as sums of outer products, a piece of rows at a time
        p = slice(at, at + (1 << 14))
        W, s = w[of[p]].double(), slice(150 + at, min(150 + at + (1 << 14), R - 200))
        terms = X[p, :, None] * W
        close(y[s], terms.sum(1), 2 * U * I * terms.abs().sum(1), dtype, "y")
        terms = D[p, None, :] * W
        close(dx[s], terms.sum(2), 2 * U * O * terms.abs().sum(2), dtype, "dx")
        terms = X[p, :, None] * D[p, None, :]
        want.index_add_(0, of[p], terms)
        size.index_add_(0, of[p], terms.abs())
    rows = (b[1:] - b[:-1]).clamp(min=1).double()[:, None, None]
    close(dw, want, 2 * U * rows * size, dtype, "dw")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_many_offsets_out_of_order_touch_nothing_outside(kind):
    R, E, I, O = 6000, 700, 24, 40
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    b = torch.randint(-100, R + 100, (E + 1,), generator=g, device=DEV)
    b[::50] = 2 ** 40
    x, w, dy = (torch.ones(*s, dtype=TYPES[kind], device=DEV) for s in ((R, I), (E, I, O), (R, O)))
    y, c1 = guarded((R, O), TYPES[kind])
    dx, c2 = guarded((R, I), TYPES[kind])
    G.spmm_segment_product(x, w, b, y)
    G.spmm_segment_product_dx(dy, w, b, dx)
    torch.cuda.synchronize()
    c1(), c2()


def test_time_of_a_million_segments():
    """A million segments of one row.  Each of the 2^20 tiles costs less than a
    microsecond of its unit's time for its place and its few kilobytes, on 256
    units a hundredth of a second in all; counting all segments for each tile
    would take 2^20 * 2^20 / 64 loads."""
    E, n = 1 << 20, 8
    x = torch.randn(E, n, device=DEV).to(torch.bfloat16)
    w = torch.randn(E, n, n, device=DEV).to(torch.bfloat16)
    b = torch.arange(E + 1, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    G.spmm_segment_product(x, w, b, y)
    G.spmm_segment_product_dx(x, w, b, dx)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 1000.0
    X, W = x.double(), w.double()
    close(y, (X[:, :, None] * W).sum(1), 2 * U * n * (X[:, :, None] * W).abs().sum(1), torch.bfloat16, "y")
    close(dx, (X[:, None, :] * W).sum(2), 2 * U * n * (X[:, None, :] * W).abs().sum(2), torch.bfloat16, "dx")
