"""Dropout: the mask against the generator on the host, values against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_rows import TYPES, close, guarded, normal, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

SEEDS = [0, 1, -1, 2 ** 62 + 12345, -2 ** 63]


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(), (1,), (3,), (4,), (5,), (8,), (9,), (7, 13), (64, 64), (3, 5, 257), (1000, 1001), (0, 4)])
def test_values_and_gradients(shape, residual, kind):
    """One product with 1 / (1 - p), which is rounded to fp32, and one sum."""
    log(f"dropout {shape} {kind} residual={residual}")
    dtype, g = TYPES[kind], rng(*(shape or (2,)))
    x, r, dy = (normal(g, *(shape or (1,)), dtype=dtype).view(shape) for _ in range(3))
    for p, seed, offset in ((0.3, SEEDS[len(shape)], 0), (0.5, 77, 2 ** 40 + 1), (0.999, 78, -3)):
        leaves = [t.to(DEV).requires_grad_() for t in ([x, r] if residual else [x])]
        s = torch.tensor([seed], device=DEV)
        y = G.dropout(leaves[0], p, s, offset, leaves[1] if residual else None)
        grads = torch.autograd.grad(y, leaves, dy.to(DEV))
        keep = rows64.kept(x.numel(), p, seed, offset).view(shape).double()
        for got, source, add in ((y, x, r if residual else None), (grads[0], dy, None)):
            term = source.double() * keep / (1 - p)
            want = term if add is None else term + add.double()
            close(got.detach(), want, rows64.U * (2 * term.abs() + (want.abs() if residual else 0)), dtype, f"p={p}")
            if add is None:
                assert bool((got.detach().cpu().double()[keep == 0] == 0).all())
        if residual:
            assert torch.equal(grads[1], dy.to(DEV))
        with torch.no_grad():
            assert torch.equal(G.dropout(leaves[0], p, s, offset, leaves[1] if residual else None), y.detach())


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_keeps_all_and_none(kind):
    x = normal(rng(1), 33, 7, dtype=TYPES[kind]).to(DEV)
    x[3] = float("nan")
    assert torch.equal(G.dropout(x, 0.0, 5)[:3], x[:3])
    assert not bool(G.dropout(x, 1.0, 5).any())
    assert torch.equal(G.dropout(x, 1.0, 5, residual=x[:1].expand(33, 7)), x[:1].expand(33, 7))
    # p next to 0 and 1 rounds to the nearest of 2^32 shares
    assert torch.equal(G.dropout(x, 1e-11, 5)[:3], x[:3])
    assert not bool(G.dropout(x, 1 - 1e-11, 5).any())


def test_dropped_elements_reach_nothing():
    p, seed = 0.4, 9
    keep = rows64.kept(4099, p, seed, 0)
    x = normal(rng(2), 4099)
    clean = G.dropout(x.to(DEV), p, seed)
    x[~keep] = float("nan")
    assert torch.equal(G.dropout(x.to(DEV), p, seed), clean)


def test_the_mask_depends_on_the_elements_number_alone():
    """Types, shapes, alignment and parts of a call agree on who is dropped."""
    n, p, seed = 100003, 0.37, 123456789
    keep = rows64.kept(n, p, seed, 4).to(DEV)
    for dtype in TYPES.values():
        assert torch.equal(G.dropout(torch.ones(n, dtype=dtype, device=DEV), p, seed, 4) != 0, keep)
        moved = torch.ones(n + 5, dtype=dtype, device=DEV)[5:]
        y, untouched = guarded((n,), dtype)
        G.spmm_dropout(moved, None, y, p, torch.tensor([seed], device=DEV), 4)
        assert torch.equal(y != 0, keep)
        untouched()
    square = torch.ones(97, 1031, device=DEV)
    assert torch.equal((G.dropout(square.t().contiguous().t(), p, seed, 4) != 0).reshape(-1).cpu(),
                       rows64.kept(97 * 1031, p, seed, 4))


def test_shares_seeds_and_offsets():
    n = 1 << 20
    one = torch.ones(n, device=DEV)
    for p in (0.1, 0.5, 0.9):
        share = float((G.dropout(one, p, 3) != 0).double().mean())
        assert abs(share - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5
    masks = [G.dropout(one, 0.5, s, o) != 0 for s, o in ((3, 0), (4, 0), (3, 1), (3 + 2 ** 32, 0), (3, 2 ** 32))]
    for i, a in enumerate(masks):
        for b in masks[:i]:
            assert abs(float((a == b).double().mean()) - 0.5) < 6 * 0.5 / n ** 0.5


def test_element_numbers_past_2_32():
    n, p, seed = (1 << 32) + 4101, 0.25, 31
    y = G.dropout(torch.ones(n, dtype=torch.bfloat16, device=DEV), p, seed)
    tail = torch.ones(5000, dtype=torch.bool)
    first = n - 5000
    at = torch.arange(first // 4, (n + 3) // 4)
    c = torch.zeros(at.numel(), 4, dtype=torch.int64)
    c[:, 0], c[:, 1] = at & rows64.MASK, at >> 32
    words = rows64.philox(c.numpy().astype("uint64"), seed, 0).reshape(-1)[first % 4:][:5000]
    tail = torch.from_numpy(words >= round(p * 2 ** 32))
    assert torch.equal(y[first:].cpu() != 0, tail)
    assert torch.equal(y[:5000].cpu() != 0, rows64.kept(5000, p, seed, 0))


def test_a_seed_that_changes_before_the_backward_pass_raises():
    x, seed = torch.ones(64, device=DEV, requires_grad=True), torch.tensor([5], device=DEV)
    y = G.dropout(x, 0.5, seed)
    seed.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
