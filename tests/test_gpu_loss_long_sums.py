"""The loss's fp32 sums over many classes or rows, however the rows lie in memory.

Sums of like terms: a chain of n equal additions rounds the same way at each of them,
so it is off by up to about n / 4 half steps (U = 2^-24) of its value, far more than sums of
random terms are.  Runs of 2,048 that are added up at their ends may be off by
2 U * 2048 / 2 for a run (the matrix cores may truncate; the partial sums of like terms
average half of the whole), 2 U for each of the n / 2048 runs' additions, and what the
terms themselves are off by, `terms`: an exponential, a quotient and the logits'
own rounding, below 64 U for the small logits here.  One chain over 32,768 terms misses
that by a factor of two and more."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.rows64 import U  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

RUN, TERMS = 2048, 64


def moved(t, shift):
    """t at an address that is `shift` elements off its own alignment."""
    whole = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
    at = whole[shift:].view(t.shape)
    at.copy_(t)
    return at


def within(got, want, n, what):
    worst = float(((got.double() - want).abs() / want.abs().clamp(min=1e-300)).max()) / U
    may = RUN + 2 * n / RUN + TERMS
    log(f"{what}: {n} terms, off by {worst:.0f} half steps at most, {may:.0f} allowed")
    assert worst <= may


@pytest.mark.parametrize("shift", [0, 1])
def test_weights_gradient_over_many_rows(shift):
    """65,536 equal rows of 4096: dw_v = R p_v g x for every class but the rows' own."""
    R, I, V = 65536, 4096, 2048
    g = torch.Generator(device=DEV).manual_seed(1)
    row = 1.0 + torch.rand(I, generator=g, device=DEV)
    x = moved(row.expand(R, I), shift).requires_grad_()
    w = moved(torch.randn(V, I, generator=g, device=DEV) * 2.0 ** -9, shift).requires_grad_()
    loss = G.linear_cross_entropy(x, w, torch.zeros(R, dtype=torch.int64, device=DEV), "sum")
    dw, = torch.autograd.grad(loss, w, torch.tensor(0.7, device=DEV))
    logits = w.detach().double() @ row.double()
    p = torch.softmax(logits, 0)
    weight = R * p * float(torch.tensor(0.7))
    # what a logit is off by, 2 I U of its magnitudes at worst, counts in all terms alike
    spread = w.detach().double().abs() @ row.double()
    terms = 2 * I * U * float(spread.max())
    want = weight[1:, None] * row.double()[None]
    worst = float(((dw[1:].double() - want).abs() / want).max())
    log(f"{R} rows at {shift}: off by {worst / U:.0f} half steps at most")
    assert worst <= (RUN + 2 * R / RUN + TERMS) * U + 2 * 2.0 ** -10 * terms


@pytest.mark.parametrize("shift", [0, 1])
def test_rows_gradient_over_many_classes(shift):
    """32,768 equal classes but the row's own, which is zero: dx = (1 - p_0) g c."""
    R, I, V = 4096, 2048, 32768
    g = torch.Generator(device=DEV).manual_seed(2)
    c = 1.0 + torch.rand(I, generator=g, device=DEV)
    w = c.expand(V, I).clone()
    w[0] = 0.0
    w = moved(w, shift).requires_grad_()
    x = moved(torch.randn(R, I, generator=g, device=DEV) * 2.0 ** -20, shift).requires_grad_()
    loss = G.linear_cross_entropy(x, w, torch.zeros(R, dtype=torch.int64, device=DEV), "sum")
    dx, = torch.autograd.grad(loss, x, torch.tensor(0.7, device=DEV))
    other = x.detach().double() @ c.double()            # the logit of every class but the first, whose is 0
    share = (V - 1) / ((V - 1) + torch.exp(-other))
    within(dx, (share * float(torch.tensor(0.7)))[:, None] * c.double()[None], V, f"dx at {shift}")


def test_sums_in_runs_and_in_one_agree_on_the_rest():
    """Unaligned rows give what aligned ones do within both ones' rounding, at sizes
    whose last run is short, one step, or not whole steps."""
    for R, I, V in ((2049, 40, 2100), (4096 + 17, 33, 300), (6145, 8, 2048 + 3)):
        g = torch.Generator(device=DEV).manual_seed(R)
        x, w = torch.randn(R, I, generator=g, device=DEV), torch.randn(V, I, generator=g, device=DEV) * I ** -0.5
        target = torch.randint(-1, V, (R,), generator=g, device=DEV)
        live = (target >= 0)[:, None]
        wd, xd = w.double(), torch.where(live, x.double(), torch.zeros((), dtype=torch.float64, device=DEV))
        d = torch.softmax(x.double() @ wd.t().contiguous(), 1)
        d[torch.arange(R, device=DEV), target.clamp(min=0)] -= 1
        d = torch.where(live, d, torch.zeros_like(d)) / int(live.sum())
        size = d.abs()
        mag = float((x.double().abs() @ wd.abs().t().contiguous()).max())
        each = (2 * I * mag + 8 * 12 + 64) * U           # logits, exponents of up to 12, the rest of a term
        for shift in (0, 1):
            leaves = [moved(t, shift).requires_grad_() for t in (x, w)]
            loss = G.linear_cross_entropy(*leaves, target, "mean")
            dx, dw = torch.autograd.grad(loss, leaves)
            for name, got, want, most, n in (("dx", dx, d @ wd, size @ wd.abs(), V),
                                             ("dw", dw, d.t().contiguous() @ xd, size.t().contiguous() @ xd.abs(), R)):
                tol = (2 * each + 2 * (min(n, RUN) + n / RUN + 8) * U) * most + 2.0 ** -24 * want.abs()
                assert bool(((got.double() - want).abs() <= tol).all()), (name, R, I, V, shift)
