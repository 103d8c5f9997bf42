"""Row operators on more tiles than one launch has blocks (2^20): blocks take
several, and elements lie past 2^31."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log
    from tests.test_gpu_segment_paths import U, close

BLOCKS = 1 << 20


def route(T, k, E):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    return G.RowRoute(torch.randint(-1, E, (T, k), generator=g, device=DEV), E)


def test_combine_past_one_launch():
    T, N = 1100000, 2048                         # 256 threads to a row of 16-byte groups
    assert T * (N // 8) // 256 > BLOCKS
    r = route(T, 1, 3)
    rows = torch.randn(T, N, device=DEV, dtype=torch.bfloat16)
    out = G.combine(r, rows)
    log("combined")
    at = r.position[:, 0].long()
    for a in range(0, T, 100000):                # one term of weight 1: the row itself, or zeros
        p = at[a:a + 100000]
        want = torch.where((p < r.offsets[-1])[:, None], rows[p], torch.zeros((), device=DEV, dtype=rows.dtype))
        assert bool((out[a:a + 100000] == want).all())


def test_combine_gradients_past_one_launch():
    T, k, N = 2200000, 2, 136                    # a wave to a row, four rows to a block
    assert T * k // 4 > BLOCKS
    r = route(T, k, 5)
    rows, dout = torch.randn(T * k, N, device=DEV).to(torch.bfloat16), torch.randn(T, N, device=DEV).to(torch.bfloat16)
    w = torch.rand(T, k, device=DEV)
    drows, dw = torch.empty_like(rows), torch.full_like(w, float("nan"))
    G.spmm_route_combine_backward(r, rows, w, dout, drows, dw)
    log("gradients")
    kept = int(r.offsets[-1])
    for a in range(0, T * k, 400000):
        q = r.order[a:a + 400000].long()
        live = (torch.arange(a, a + q.numel(), device=DEV) < kept)[:, None]
        d = dout[q // k].float()
        zero = torch.zeros((), device=DEV)
        # one product in 32 bits, rounded once
        assert torch.equal(drows[a:a + 400000], torch.where(live, w.reshape(-1)[q, None] * d, zero).to(torch.bfloat16))
        dots = torch.where(live, rows[a:a + 400000].double() * d.double(), zero.double())
        close(dw.reshape(-1)[q], dots.sum(1), N * U * dots.abs().sum(1), torch.float32, "dweight")


def test_segment_product_past_one_launch():
    R, n = 128 * BLOCKS + 5000, 8                # 128 rows to a tile
    x = torch.randn(R, n, device=DEV)
    w = torch.randn(2, n, n, device=DEV)
    cut = 128 * BLOCKS - 77
    y = torch.full_like(x, float("nan"))
    G.spmm_segment_product(x, w, torch.tensor([0, cut, R], device=DEV), y)
    log("product")
    for a in [*range(0, R, 1 << 24), cut, R - 3000]:
        for e, (lo, hi) in enumerate(((a, min(a + 3000, cut)), (max(a, cut), min(a + 3000, R)))):
            if lo < hi:
                X, W = x[lo:hi].double(), w[e].double()
                close(y[lo:hi], X @ W, 2 * U * n * (X.abs() @ W.abs()), torch.float32, f"rows from {lo}")


def test_weight_gradients_past_one_launch():
    E, n = BLOCKS + 3000, 8                      # a tile to a segment
    x, dy = (torch.randn(E, n, device=DEV).to(torch.bfloat16) for _ in range(2))
    dw = torch.full((E, n, n), float("nan"), device=DEV, dtype=torch.bfloat16)
    G.spmm_segment_product_dw(x, dy, torch.arange(E + 1, device=DEV), dw)
    assert torch.equal(dw, (x.float()[:, :, None] * dy.float()[:, None, :]).to(torch.bfloat16))
