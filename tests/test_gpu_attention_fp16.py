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
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_attention import SLACK, bounds, on_gpu  # noqa: E402
from tests.test_gpu_rows import guarded, half_step, normal, rng  # noqa: E402

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


SHAPES = [([1], [1], 1, 1, 8), ([3, 0, 70, 1], None, 6, 2, 40), ([300, 1, 257], None, 4, 1, 72),
          ([2] * 700, None, 2, 2, 16), ([2100], None, 4, 1, 128), ([2500, 1], [40, 9], 2, 1, 96),
          ([0, 0], [5, 7], 3, 1, 24), ([1, 1], [3000, 20], 8, 2, 64)]


@pytest.mark.parametrize("rows,keys,H,Hk,D", SHAPES)
def test_workspaces_of_exactly_their_size(rows, keys, H, Hk, D):
    """The C calls with workspaces of as many bytes as they ask for, guarded: nothing
    beside them is written, and the results are the binding's."""
    g = rng(sum(rows), H, D)
    ro, ko = bounds(rows), bounds(rows if keys is None else keys)
    R, K, S = ro[-1] + 2, ko[-1] + 3, len(rows)
    q, k, v, dout = (normal(g, n, h, D, dtype=F16).to(DEV) for n, h in ((R, H), (K, Hk), (K, Hk), (R, H)))
    o, kof = torch.tensor(ro, device=DEV), torch.tensor(ko, device=DEV)
    sizes, lib = (R, K, S, H, Hk, D), G.lib()

    def workspace(call):
        n = ctypes.c_int64()
        assert getattr(lib, call)(*sizes, G.SPMM_F16, ctypes.byref(n)) == 0
        whole, untouched = guarded((max(1, n.value // 4),), torch.float32)
        return whole, n.value, untouched

    at = [t.data_ptr() for t in (q, k, v, o, kof)]
    heads = [at[0], H * D, at[1], Hk * D, at[2], Hk * D, at[3], at[4]]
    for causal in (0, 1):
        out, rest, dq = (torch.empty_like(q) for _ in range(3))
        lse, dk, dv = torch.empty(R, H, device=DEV), torch.empty_like(k), torch.empty_like(v)
        work, n, first = workspace("spmm_segment_attention_workspace")
        back, m, second = workspace("spmm_segment_attention_backward_workspace")
        stream = torch.cuda.current_stream().cuda_stream
        how = [*sizes, D ** -0.5, causal, G.SPMM_F16]
        made = [t.data_ptr() for t in (out, rest, lse)]
        grads = [t.data_ptr() for t in (dout, dq, dk, dv)]
        assert lib.spmm_segment_attention(*heads, *made, *how, work.data_ptr(), n, stream) == 0
        assert lib.spmm_segment_attention_backward(*heads, *made, *grads, *how, back.data_ptr(), m, stream) == 0
        torch.cuda.synchronize()
        first(), second()
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        same = G.segment_attention(*leaves, o, kof, causal=bool(causal))
        for a, b in zip((out, dq, dk, dv), (same, *torch.autograd.grad(same, leaves, dout))):
            assert torch.equal(a, b)


def test_captured_and_on_two_streams():
    """Forward and backward captured and replayed with gradients of other sizes and
    other offsets; two passes at once on two streams."""
    g = rng(41)
    shapes = ((400, 4), (400, 2), (400, 2))
    static = [normal(g, n, h, 64, dtype=F16).to(DEV).requires_grad_() for n, h in shapes]
    dout, o = normal(g, 400, 4, 64, dtype=F16).to(DEV), torch.tensor([0, 300, 400], device=DEV)

    def run(leaves, o, dout):
        out = G.segment_attention(*leaves, o, causal=True)
        return [out, *torch.autograd.grad(out, leaves, dout)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(static, o, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        got = run(static, o, dout)
    for rep, (size, lengths) in enumerate([(1e-4, [0, 399, 400]), (1024.0, [0, 10, 400]), (1.0, [5, 200, 390])]):
        new = [normal(g, n, h, 64, dtype=F16).to(DEV) for n, h in shapes]
        with torch.no_grad():
            for a, b in zip(static, new):
                a.copy_(b)
            dout.copy_(normal(g, 400, 4, 64, scale=size).to(F16))
            o.copy_(torch.tensor(lengths))
        float(torch.randn(1 << 18, device=DEV).sum())
        graph.replay()
        torch.cuda.synchronize()
        eager = run([t.requires_grad_() for t in new], torch.tensor(lengths, device=DEV), dout.clone())
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), f"replay {rep}"
    both, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            both.append(run([t.detach().clone().requires_grad_() for t in new], torch.tensor(lengths, device=DEV),
                            dout.clone()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in zip(*both, eager) for a in pair[:2] for b in pair[2:])
