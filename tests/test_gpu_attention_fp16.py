"""Attention in fp16 where a probability or the gradient of a score is small or
large beside fp16's own range: long segments, small and large incoming gradients,
weights far below the largest.

Bounds.  rows64 derives what every rounding may do and grants each probability and
each gradient of a score half of fp16's smallest subnormal, 2^-25, on top.  Here that
is replaced by what the kernels may lose when they hold these values times powers of
two:
* a weight times 2^12 of the largest one, or of the row's sum: 2^-37 each;
* the gradients of scores of a row (dq) times 2^12 and a power of two that brings the
  largest so far to 2^11 at least: 2^-36 of the largest each;
* those of a key (dk) times 2^12 and a power of two that brings their bound, the longest
  dout times the length of v plus the largest dout.out, to 4 at least: 2^-39 of it each;
* what out's rounding leaves off is kept in fp16 as it is: 2^-25 an element.
All of these are far below half a step of the outputs, so a comparison asks for the
outputs' own precision; each test makes sure that its bounds are a small share of the
values."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_attention import SLACK, on_gpu  # noqa: E402
from tests.test_gpu_rows import half_step, normal, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

F16 = torch.float16
WEIGHT, ROW, KEY, REST = 2.0 ** -37, 2.0 ** -36, 2.0 ** -39, 2.0 ** -25


def wanted(monkeypatch, q, k, v, causal, scale, dout):
    """(value, bound) of out, dq, dk, dv of one segment."""
    half, _ = rows64.steps(F16)
    n, m = q.shape[0], k.shape[0]
    with monkeypatch.context() as patch:
        patch.setattr(rows64, "steps", lambda dtype: (half, 0.0))
        want = rows64.attention(q, k, v, [0, n], [0, m], causal, scale, dout)
    H, group = q.shape[1], q.shape[1] // k.shape[1]
    seen = torch.ones(n, m, dtype=torch.float64)
    if causal:
        seen = (torch.arange(m)[None, :] <= torch.arange(n)[:, None] + (m - n)).double()
    more = [bound.clone() for _, bound in want]
    kept = []
    for h in range(H):
        x, y, z, g = (t.double() for t in (q[:, h], k[:, h // group], v[:, h // group], dout[:, h]))
        s = (scale * (x @ y.T)).masked_fill(seen == 0, -1e300)
        p = torch.softmax(s, 1) * seen
        lost = WEIGHT * (seen @ z.abs())
        more[0][:, h] += lost
        more[3][:, h // group] += WEIGHT * (seen.T @ g.abs())
        delta = (g.abs() * (lost + REST)).sum(1, keepdim=True)
        own = (g * want[0][0][:, h]).sum(1, keepdim=True)
        ds = (p * (g @ z.T - own)).abs()
        more[1][:, h] += scale * ((p * delta + ROW * ds.amax(1, keepdim=True) * seen) @ y.abs())
        kept.append((x, p, delta, float(g.norm(dim=1).max()), float(own.abs().max())))
    for h, (x, p, delta, _, _) in enumerate(kept):
        mates = kept[h // group * group:][:group]
        most = max(t[3] for t in mates) * v[:, h // group].double().norm(dim=1) + max(t[4] for t in mates)
        more[2][:, h // group] += scale * ((p * delta).T @ x.abs() + KEY * most[:, None] * (seen.T @ x.abs()))
    return [(value, bound) for (value, _), bound in zip(want, more)]


def check(got, want, names=("out", "dq", "dk", "dv"), share=20):
    for name, t, (value, before) in zip(("out", "dq", "dk", "dv"), got, want):
        t = t.detach().double().cpu()
        tol = SLACK * (before + half_step(value.abs() + before, F16)) + 1e-300
        worst = float(((t - value).abs() / tol).nan_to_num(float("inf")).max())
        reach = float((value.abs() / tol).max())
        log(f"  {name}: worst error {worst:.3g} of its bound, which is 1 / {reach:.3g} of the largest value")
        assert worst <= 1.0, f"{name}: error {worst:.3g} times its bound"
        assert name not in names or reach > share, f"{name}: a bound of 1 / {reach:.3g} of the value shows nothing"


def run(monkeypatch, q, k, v, dout, causal=False, scale=None, **how):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    got = on_gpu(q, k, v, dout, [0, q.shape[0]], [0, k.shape[0]], causal, scale)
    check(got, wanted(monkeypatch, q, k, v, causal, scale, dout), **how)


@pytest.mark.parametrize("m", [16384, 131072])
def test_weights_of_a_long_segment(monkeypatch, m):
    """A few rows over many keys of like weight: p is 2^-14 or 2^-17, dv = p dout with
    dout of about 2^10 is well inside fp16's range."""
    g = rng(m, 3)
    q, k = normal(g, 3, 2, 16, dtype=F16, scale=0.3), normal(g, m, 1, 16, dtype=F16)
    v, dout = normal(g, m, 1, 16, dtype=F16), normal(g, 3, 2, 16, dtype=F16, scale=1024.0)
    run(monkeypatch, q, k, v, dout, names=("dv",))


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("size", [1e-3, 1e-4])
def test_small_gradients_of_a_long_segment(monkeypatch, size, D):
    """dout of 1e-3 and 1e-4 over 32,768 keys: single gradients of scores are a few
    2^-24 or less, their sums are not.  Terms of a sum have one sign, so that the
    bounds, which add up magnitudes, are close: v and k point to +- one direction."""
    g, m = rng(int(1 / size), D), 32768
    s = torch.where(torch.rand(m, 1, 1, generator=g) < 0.5, -1.0, 1.0).double()
    a, w = (normal(g, 1, 1, D).sign().double() for _ in range(2))
    v = (0.25 * s * a + 0.02 * normal(g, m, 1, D).double()).to(F16)
    dout = (size * (a + 0.1 * normal(g, 5, 2, D).double())).to(F16)
    # dq: large keys along w, small rows
    k = (4096 * (s * w + 0.1 * normal(g, m, 1, D).double())).to(F16)
    q = normal(g, 5, 2, D, dtype=F16, scale=2.0 ** -13)
    run(monkeypatch, q, k, v, dout, names=("dq",))
    # dk: large rows along w, small keys
    k = normal(g, m, 1, D, dtype=F16, scale=2.0 ** -13)
    q = (4096 * (w + 0.1 * normal(g, 5, 2, D).double())).to(F16)
    run(monkeypatch, q, k, v, dout, names=("dk",))


@pytest.mark.parametrize("keys", [2, 200, 700])
@pytest.mark.parametrize("D", [64, 128])
def test_large_gradients(monkeypatch, D, keys):
    """Gradients of scores far above 65,504 whose sums times k and q are not."""
    g, half = rng(D, keys), keys // 2
    a = normal(g, 1, 1, D).sign()
    s = torch.ones(keys, 1, 1)
    s[half:] = -1.0
    v = (64.0 * s * a).to(F16)
    dout = (1024.0 * (a + 0.1 * normal(g, 3, 1, D))).to(F16)
    k = (2.0 ** -8 * (s * a + 0.1 * normal(g, keys, 1, D))).to(F16)
    q = normal(g, 3, 1, D, dtype=F16, scale=2.0 ** -8)
    run(monkeypatch, q, k, v, dout, scale=0.125, names=("dq", "dv"))


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("m", [40, 300, 5000])
def test_gradients_of_values_of_small_weight(monkeypatch, m, D):
    """One key has nearly all the weight, the others 2^-22 and 2^-24.4 of it: their dv is
    p dout, with dout of about 2^13 far above fp16's smallest numbers."""
    g = rng(m, D, 5)
    q, k = torch.zeros(2, 2, D, dtype=F16), torch.zeros(m, 1, D, dtype=F16)
    q[..., 0] = 1.0
    k[:, 0, 0] = torch.where(torch.rand(m, generator=g) < 0.5, -22.0, -24.4) * 0.6931
    k[m // 3] = 0.0
    v, dout = normal(g, m, 1, D, dtype=F16), (8192.0 * (1.0 + 0.1 * normal(g, 2, 2, D))).to(F16)
    run(monkeypatch, q, k, v, dout, scale=1.0, names=("out", "dv"))


def test_weights_far_below_the_largest(monkeypatch):
    """Every 256th key has nearly all the weight and no value; the others weigh about
    2^-22.7 of it and make up all of out."""
    g, m = rng(77), 65536
    k = torch.zeros(m, 1, 8, dtype=F16)
    k[::256, 0, 0] = 22.7 * 0.6931                     # 22.7 in base 2
    q = torch.zeros(1, 2, 8, dtype=F16)
    q[..., 0] = 1.0
    v = (1024.0 * (1.0 + 0.1 * normal(g, m, 1, 8))).to(F16)
    v[::256] = 0.0
    run(monkeypatch, q, k, v, normal(g, 1, 2, 8, dtype=F16), scale=1.0, names=("out",))


@pytest.mark.parametrize("n,m", [(20, 25), (90, 120), (300, 310), (700, 900)])
@pytest.mark.parametrize("D", [24, 40, 64, 72, 128])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_gradients_of_scores_of_any_size(monkeypatch, order, D, n, m):
    """Values whose size rises or falls by 2^14 from the first key to the last, and
    incoming gradients that do by 2^10 from the first row: what holds the gradients of
    scores has to follow, for rows and for keys, in every kind of tile."""
    g = rng(n, m, D, len(order))
    size = torch.linspace(-7, 7, m), torch.linspace(-5, 5, n)
    if order == "falling":
        size = size[0].flip(0), size[1].flip(0)
    if order == "mixed":
        size = size[0][torch.randperm(m, generator=g)], size[1][torch.randperm(n, generator=g)]
    q, k = normal(g, n, 2, D, dtype=F16), normal(g, m, 1, D, dtype=F16)
    v = (normal(g, m, 1, D) * torch.exp2(size[0])[:, None, None]).to(F16)
    dout = (normal(g, n, 2, D) * torch.exp2(size[1])[:, None, None]).to(F16)
    for causal in (False, True):
        run(monkeypatch, q, k, v, dout, causal, share=4)


def test_zero_and_infinite_gradients():
    """No gradient at all gives zeros; an infinite one stays with its row and keys."""
    g = rng(3, 9)
    q, k, v = (normal(g, 90, 1, 64, dtype=F16) for _ in range(3))
    dout = torch.zeros(90, 1, 64, dtype=F16)
    ro = [0, 40, 90]
    got = on_gpu(q, k, v, dout, ro, ro, True)
    assert not any(bool(t.any()) for t in got[1:])
    dout[60, 0, 5] = float("inf")
    got = on_gpu(q, k, v, dout, ro, ro, True)
    assert all(bool(torch.isfinite(t[:40]).all()) for t in got[1:])
    assert not bool(torch.isfinite(got[1][60]).any()) and not bool(got[1][40:60].any())


def test_wide_rows_of_joined_parts_follow_the_same_bits():
    """The call without gradients, and gradients one at a time, give the same bits."""
    g = rng(6, 6)
    q, k, v = (normal(g, 2, 4, 64, dtype=F16), normal(g, 9000, 1, 64, dtype=F16), normal(g, 9000, 1, 64, dtype=F16))
    dout = normal(g, 2, 4, 64, dtype=F16, scale=1e-3)
    o, ko = torch.tensor([0, 2], device=DEV), torch.tensor([0, 9000], device=DEV)
    got = on_gpu(q, k, v, dout, [0, 2], [0, 9000], False)
    with torch.no_grad():
        assert torch.equal(G.segment_attention(q.to(DEV), k.to(DEV), v.to(DEV), o, ko), got[0].detach())
    for i in range(3):
        leaves = [t.to(DEV) for t in (q, k, v)]
        leaves[i].requires_grad_()
        out = G.segment_attention(*leaves, o, ko)
        assert torch.equal(torch.autograd.grad(out, leaves[i], dout.to(DEV))[0], got[1 + i])
