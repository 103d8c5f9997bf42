"""Attention within segments against its plain form in 64 bits (tests/rows64.py,
which derives the tolerances)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_rows import TYPES, guarded, half_step, normal, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

SLACK = 1.02


def close(got, want, dtype, what):
    value, before = want
    got = got.detach().double().cpu()
    tol = SLACK * (before + half_step(value.abs() + before, dtype)) + 1e-300
    bad = ~((got - value).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error "
                           f"{float((got - value).abs().max()):.3e}, worst ratio "
                           f"{float(((got - value).abs() / tol).max()):.3g}")


def bounds(lengths, first=0):
    return [first + int(n) for n in np.cumsum([0] + list(lengths))]


def case(rows, keys, H, Hk, D, dtype, front=0, back=0, seed=0):
    """q, k, v, dout with NaN and infinities in the rows outside the segments."""
    g = rng(sum(rows), H, D, seed)
    ro = bounds(rows, front)
    ko = ro if keys is None else bounds(keys, front)
    R, K = ro[-1] + back, ko[-1] + back
    q, dout = normal(g, R, H, D, dtype=dtype, scale=1.5), normal(g, R, H, D, dtype=dtype)
    k, v = normal(g, K, Hk, D, dtype=dtype), normal(g, K, Hk, D, dtype=dtype)
    for t, o in ((q, ro), (dout, ro), (k, ko), (v, ko)):
        t[:o[0]] = float("nan")
        t[o[-1]:] = float("inf")
    return q, k, v, dout, ro, ko


def on_gpu(q, k, v, dout, ro, ko, causal, scale=None, keys=True):
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    offsets = torch.tensor(ro, device=DEV)
    out = G.segment_attention(*leaves, offsets, torch.tensor(ko, device=DEV) if keys else None, causal=causal, scale=scale)
    return [out, *torch.autograd.grad(out, leaves, dout.to(DEV))]


def compare(rows, keys, H, Hk, D, kind, causal, front=0, back=0, scale=None):
    log(f"attention rows={rows if len(rows) < 12 else len(rows)} keys={keys if keys is None or len(keys) < 12 else '..'} "
        f"H={H}/{Hk} D={D} {kind} causal={causal}")
    dtype = TYPES[kind]
    q, k, v, dout, ro, ko = case(rows, keys, H, Hk, D, dtype, front, back)
    got = on_gpu(q, k, v, dout, ro, ko, causal, scale, keys is not None)
    want = rows64.attention(q, k, v, ro, ko, causal, D ** -0.5 if scale is None else scale, dout)
    for name, t, w in zip(("out", "dq", "dk", "dv"), got, want):
        close(t, w, dtype, name)
    with torch.no_grad():                               # the call without gradients
        only = G.segment_attention(*(t.to(DEV) for t in (q, k, v)), torch.tensor(ro, device=DEV),
                                   torch.tensor(ko, device=DEV), causal=causal, scale=scale)
    assert torch.equal(only, got[0].detach())


# around every border of tiles: 32 and 128 rows or keys, 32 and 64 to a step
LENGTHS = [([1], None), ([2, 1, 3], None), ([31, 32, 33], None), ([63, 64, 65, 1, 0, 2], None), ([127, 128, 129], None),
           ([0, 0, 5, 0], None), ([300, 1, 257], None), ([0], None),
           ([1, 1, 1], [1, 40, 333]), ([1, 2], [2000, 1]), ([5, 0, 7, 3], [0, 9, 70, 129]), ([40, 200, 3], [20, 133, 0]),
           ([260], [32]), ([3], [700])]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows,keys", LENGTHS)
def test_lengths(rows, keys, kind, causal):
    compare(rows, keys, 4, 2, 40, kind, causal, front=3, back=4)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("D", [1, 3, 7, 8, 16, 31, 32, 33, 48, 64, 65, 72, 96, 97, 100, 120, 127, 128])
def test_widths(D, kind):
    compare([37, 140], None, 2, 1, D, kind, True)
    compare([150], [90], 1, 1, D, kind, False, back=1)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (7, 1), (14, 2), (8, 1), (64, 2), (130, 1)])
def test_grouped_heads(H, Hk, kind):
    compare([9, 70], None, H, Hk, 24, kind, True, back=2)
    compare([1, 1], [150, 8], H, Hk, 24, kind, True)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_few_rows_of_long_segments_and_the_reverse(kind):
    """Keys in parts that are joined, and rows in parts that are added."""
    compare([1, 2, 1], [3000, 700, 5000], 4, 1, 64, kind, True)
    compare([1], [9000], 2, 2, 128, kind, False)
    compare([2500, 3001], [40, 90], 2, 1, 96, kind, False)
    compare([2100], None, 4, 1, 128, kind, True)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("S", [62, 63, 64, 65, 200, 4100])
def test_many_segments(S, kind):
    g = np.random.default_rng(S)
    n = g.integers(0, 40 if S < 1000 else 6, S)
    n[g.integers(0, S, 5)] = 0
    compare(list(n), None, 2, 2, 16, kind, False, front=1, back=1)
    if S < 100:
        compare(list(n), list(g.integers(0, 50, S)), 2, 1, 16, kind, True)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_scales(kind):
    for scale in (1e-4, 0.5, 3.0):
        compare([70, 33], None, 2, 1, 32, kind, True, scale=scale)


def test_scores_at_the_ends_of_fp32():
    """The lowest and highest scores that stay finite: the running maximum takes
    them, and a row of equal scores averages v."""
    q = torch.full((3, 1, 4), 2.0 ** 60)
    k = torch.full((70, 1, 4), -2.0 ** 60)
    v = normal(rng(5), 70, 1, 4)
    q[1] = -q[1]
    q[2] = 0.0
    o = torch.tensor([0, 3], device=DEV)
    out = G.segment_attention(q.to(DEV), k.to(DEV), v.to(DEV), o, torch.tensor([0, 70], device=DEV), scale=1.0)
    want = v.double().mean(0).expand(3, 1, 4)
    assert float((out.double().cpu() - want).abs().max()) <= 70 * 4 * rows64.U * float(v.abs().max())
    k[33] *= 2                                          # one key further down or up decides
    out = G.segment_attention(q.to(DEV), k.to(DEV), v.to(DEV), o, torch.tensor([0, 70], device=DEV), scale=1.0)
    assert torch.equal(out[1].cpu(), v[33])
    rest = torch.cat([v[:33], v[34:]]).double().mean(0)
    assert float((out[0].double().cpu() - rest).abs().max()) <= 70 * 4 * rows64.U * float(v.abs().max())


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_parts_of_a_wider_row_are_read_in_place(kind):
    """q, k and v as views of one projection, and such views with odd strides,
    give the same bits as packed copies."""
    g, dtype = rng(31), TYPES[kind]
    for H, Hk, D, extra in ((4, 2, 64, 0), (2, 2, 40, 8), (2, 1, 33, 3)):
        wide = normal(g, 200, (H + 2 * Hk) * D + extra, dtype=dtype).to(DEV).requires_grad_()
        o = torch.tensor([0, 90, 200], device=DEV)
        dout = normal(g, 200, H, D, dtype=dtype).to(DEV)

        def parts(t):
            q, k, v, _ = t.split([H * D, Hk * D, Hk * D, extra], 1)
            return q.unflatten(1, (H, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))

        out = G.segment_attention(*parts(wide), o, causal=True)
        dwide, = torch.autograd.grad(out, wide, dout)
        packed = [t.detach().contiguous().requires_grad_() for t in parts(wide)]
        same = G.segment_attention(*packed, o, causal=True)
        grads = torch.autograd.grad(same, packed, dout)
        assert torch.equal(out, same)
        assert all(torch.equal(a, b) for a, b in zip(parts(dwide), grads))
        turned = [t.detach().transpose(0, 1).contiguous().transpose(0, 1) for t in parts(wide)]   # heads outermost
        assert torch.equal(G.segment_attention(*turned, o, causal=True), same)
        # broadcast heads: their gradients are added up by torch
        one = wide.detach()[:, :D].unsqueeze(1).clone().requires_grad_()
        out = G.segment_attention(one.expand(200, H, D), packed[1], packed[2], o)
        assert torch.autograd.grad(out, one, dout)[0].shape == one.shape


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_any_alignment_and_guarded_outputs(kind, shift):
    dtype, g = TYPES[kind], rng(8, shift)
    R, H, Hk, D = 75, 2, 1, 64

    def at(t):
        whole = torch.zeros(t.numel() + shift + 40, dtype=dtype, device=DEV)
        whole[shift:shift + t.numel()] = t.reshape(-1).to(DEV)
        return whole[shift:shift + t.numel()].view(t.shape)

    q, k, v, dout = (normal(g, R, h, D, dtype=dtype) for h in (H, Hk, Hk, H))
    o = torch.tensor([2, 40, 70], device=DEV)
    out, a = guarded((R, H, D), dtype)
    rest, b = guarded((R, H, D), dtype)
    lse, c = guarded((R, H), torch.float32)
    dq, d = guarded((R, H, D), dtype)
    dk, e = guarded((R, Hk, D), dtype)
    dv, f = guarded((R, Hk, D), dtype)
    qa, ka, va, da = (at(t) for t in (q, k, v, dout))
    G.spmm_segment_attention(qa, ka, va, o, o, out, lse, True, 0.125, rest)
    G.spmm_segment_attention_backward(qa, ka, va, o, o, out, lse, da, dq, dk, dv, True, 0.125, rest)
    want = rows64.attention(q, k, v, o.tolist(), o.tolist(), True, 0.125, dout)
    for name, t, w in zip(("out", "dq", "dk", "dv"), (out, dq, dk, dv), want):
        close(t, w, dtype, name)
    for untouched in (a, b, c, d, e, f):
        untouched()
    # gradients that are not asked for
    only, g1 = guarded((R, Hk, D), dtype)
    G.spmm_segment_attention_backward(qa, ka, va, o, o, out, lse, da, None, None, only, True, 0.125, rest)
    assert torch.equal(only, dv)
    G.spmm_segment_attention_backward(qa, ka, va, o, o, out, lse, da, None, only, None, True, 0.125, rest)
    assert torch.equal(only, dk)
    g1()


def test_offsets_out_of_range_and_out_of_order_stay_inside():
    g, H, D = rng(12), 2, 32
    q, k, v, dout = (normal(g, 100, H, D).to(DEV) for _ in range(4))
    for ro, ko in (([-5, 40, 300], [0, 50, 2 ** 40]), ([60, 20, 90], [0, 70, 10]), ([200, 300, 400], [-9, -7, -1])):
        ro, ko = torch.tensor(ro, device=DEV), torch.tensor(ko, device=DEV)
        out, a = guarded((100, H, D), torch.float32, 0.0)
        lse, b = guarded((100, H), torch.float32, 0.0)
        grads = [guarded((100, H, D), torch.float32, 0.0) for _ in range(3)]
        G.spmm_segment_attention(q, k, v, ro, ko, out, lse)
        G.spmm_segment_attention_backward(q, k, v, ro, ko, out, lse, dout, *(t for t, _ in grads))
        torch.cuda.synchronize()
        a(), b()
        for _, untouched in grads:
            untouched()
    # out of range alone: as if cut to the rows
    got = G.segment_attention(q, k, v, torch.tensor([-5, 40, 300], device=DEV), torch.tensor([0, 50, 2 ** 40], device=DEV))
    want = G.segment_attention(q, k, v, torch.tensor([0, 40, 100], device=DEV), torch.tensor([0, 50, 100], device=DEV))
    assert torch.equal(got, want)


def test_infinite_values_spread_within_their_segment_alone():
    g, o = rng(13), torch.tensor([0, 40, 80], device=DEV)
    q, k, v, dout = (normal(g, 80, 1, 32).to(DEV) for _ in range(4))
    clean = G.segment_attention(q, k, v, o)
    for t in (q, k, v):
        t[50] = float("nan")
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out = G.segment_attention(*leaves, o)
    assert torch.equal(out[:40], clean[:40]) and bool(torch.isnan(out[40:]).all())
    for d in torch.autograd.grad(out, leaves, dout):
        assert bool(torch.isfinite(d[:40]).all()) and bool(torch.isnan(d[40:]).any())


def test_element_offsets_past_2_32():
    """Two rows against the ends of keys of 2^32 elements and more."""
    K, Hk, D = 270001, 128, 128
    g = torch.Generator(device=DEV).manual_seed(5)
    k = torch.randn(K, Hk, D, dtype=torch.bfloat16, generator=g, device=DEV)
    v = torch.randn(K, Hk, D, dtype=torch.bfloat16, generator=g, device=DEV)
    q = torch.randn(2, Hk, D, dtype=torch.bfloat16, generator=g, device=DEV)
    assert k.numel() > 2 ** 32
    ko = torch.tensor([0, K - 700, K], device=DEV)
    out = G.segment_attention(q, k, v, torch.tensor([0, 1, 2], device=DEV), ko, causal=True)
    h = 77                                              # a head alone, the last segment alone
    want = rows64.attention(q[1:, h:h + 1].cpu(), k[K - 700:, h:h + 1].cpu(), v[K - 700:, h:h + 1].cpu(), [0, 1],
                            [0, 700], True, D ** -0.5)
    close(out[1:, h:h + 1], want[0], torch.bfloat16, "out")
    long = rows64.attention(q[:1, h:h + 1].cpu(), k[:K - 700, h:h + 1].cpu(), v[:K - 700, h:h + 1].cpu(), [0, 1],
                            [0, K - 700], True, D ** -0.5)
    close(out[:1, h:h + 1], long[0], torch.bfloat16, "out")


def test_two_runs_give_the_same_bits():
    q, k, v, dout, ro, ko = case([700, 1500, 40], None, 8, 2, 128, torch.bfloat16)
    runs = [on_gpu(q, k, v, dout, ro, ko, True) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_gradients_against_differences():
    """<gradient, v> against (f(p + h v) - f(p - h v)) / 2 h of the kernels' own
    forward, f = sum(c out), in fp32.  What the difference leaves out is taken from
    64 bits, where it is the difference less the derivative; what is left is f's
    rounding on both sides, which rows64 bounds, over 2 h.  The directions have the
    signs of the exact gradient, so that slopes add up and stand out of the bound."""
    q, k, v, c, ro, ko = case([20, 45], [33, 60], 2, 1, 16, torch.float32)
    p, h = [q, k, v], 2.0 ** -6
    grads = on_gpu(q, k, v, c, ro, ko, True)[1:]
    exact = rows64.attention(q, k, v, ro, ko, True, 0.25, c)[1:]
    g = rng(99)
    for i in range(3):
        step = normal(g, *p[i].shape).abs() * exact[i][0].sign().float()
        ends = [p[i] + h * step, p[i] - h * step]
        moved = (ends[0].double() - ends[1].double()) / (2 * h)
        f, f64, err = [], [], 0.0
        for e in ends:
            at = [e if j == i else t for j, t in enumerate(p)]
            out = G.segment_attention(*(t.to(DEV) for t in at), torch.tensor(ro, device=DEV),
                                      torch.tensor(ko, device=DEV), causal=True)
            value, bound = rows64.attention(*at, ro, ko, True, 0.25)[0]
            f.append(float((c.double() * out.double().cpu()).sum()))
            f64.append(float((c.double() * value).sum()))
            err += float((c.double().abs() * (bound + half_step(value.abs() + bound, torch.float32))).sum())
        value, bound = exact[i]
        left_out = (f64[0] - f64[1]) / (2 * h) - float((value * moved).sum())
        slope = float((grads[i].double().cpu() * moved).sum())
        tol = SLACK * (err / (2 * h) + float((moved.abs() * (bound + half_step(value.abs() + bound, torch.float32))).sum()))
        assert abs(slope + left_out - (f[0] - f[1]) / (2 * h)) <= tol
        assert tol < 0.02 * abs(slope)
