"""Attention and the loss where element offsets pass 2^31 and 2^32.  Inputs are made so
that single far rows decide what is compared: a result of other rows cannot pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_attention import close  # noqa: E402
from tests.test_gpu_rows import TYPES, half_step, normal, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

BF16 = torch.bfloat16
ROWS, HEADS, WIDTH = 270001, 128, 128                  # 4.4e9 elements


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def test_far_keys_decide():
    """One row against 270,001 keys, cut into parts: zeros but for a few, each of which
    has nearly all the weight of one head."""
    k = torch.zeros(ROWS, HEADS, WIDTH, dtype=BF16, device=DEV)
    v = torch.zeros(ROWS, HEADS, WIDTH, dtype=BF16, device=DEV)
    q = torch.zeros(1, HEADS, WIDTH, dtype=BF16, device=DEV)
    q[..., 0] = 1.0
    g = torch.Generator().manual_seed(8)
    # 2^31 elements are at row 131,072, 2^32 at 262,144
    fixed = [0, 63, 64, 131071, 131072, 131073, 262143, 262144, 262145, ROWS - 65, ROWS - 2, ROWS - 1]
    at = torch.cat([torch.tensor(fixed), torch.randint(0, ROWS, (HEADS - len(fixed),), generator=g)]).to(DEV)
    h = torch.arange(HEADS, device=DEV)
    value = normal(g, HEADS, WIDTH, dtype=BF16).to(DEV)
    k[at, h, 0] = 40.0
    v[at, h] = value
    ko = torch.tensor([0, ROWS], device=DEV)
    out = G.segment_attention(q, k, v, torch.tensor([0, 1], device=DEV), ko, scale=1.0)
    # the others' weight together is 270,000 e^-40, nothing beside a rounding
    assert torch.equal(out[0], value)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    dout = normal(g, 1, HEADS, WIDTH, dtype=BF16).to(DEV)
    out = G.segment_attention(*leaves, torch.tensor([0, 1], device=DEV), ko, scale=1.0)
    dq, dk, dv = torch.autograd.grad(out, leaves, dout)
    assert torch.equal(dv[at, h], dout[0])
    total = sum(float(dv[a:a + 20000].float().abs().sum(dtype=torch.float64)) for a in range(0, ROWS, 20000))
    most = float(dout.float().abs().sum(dtype=torch.float64))
    assert abs(total - most) <= 1e-3 * most
    assert bool(torch.isfinite(dq).all()) and float(dk.abs().max()) < 1e-2


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("K", [3000, 20000, 270001])
def test_every_part_of_a_long_segment_counts(K, kind):
    """One row against keys that are cut into parts and joined: 101 keys, spread over all
    of them, have equal weight and the rest none (e^-80), so out is the mean of their values
    and dv a 101st of dout.  One of them amiss moves out by about a hundredth of a value,
    which is ten times what the bound allows: half a step of the type on a mean of about
    a tenth, and 2 * 101 u of the sum of magnitudes for the additions, the quotient and
    the joins (weights of 1 are exact in every type)."""
    dtype, H, Hk, D, n = TYPES[kind], 4, 2, 64, 101
    g = rng(K, len(kind))
    at = torch.linspace(0, K - 1, n).long()
    k, v = torch.zeros(K, Hk, D, dtype=dtype), normal(g, K, Hk, D, dtype=dtype)
    k[at, :, 0] = 80.0
    q = torch.zeros(1, H, D, dtype=dtype)
    q[..., 0] = 1.0
    dout = normal(g, 1, H, D, dtype=dtype)
    leaves = [t.to(DEV).requires_grad_() for t in (q, k, v)]
    out = G.segment_attention(*leaves, torch.tensor([0, 1], device=DEV), torch.tensor([0, K], device=DEV), scale=1.0)
    mean = v[at].double().mean(0).repeat_interleave(H // Hk, 0)[None]
    size = v[at].double().abs().mean(0).repeat_interleave(H // Hk, 0)[None]
    before = (2 * n + 8) * 2.0 ** -24 * size
    close(out, (mean, before), dtype, "out")
    dv = torch.autograd.grad(out, leaves[2], dout.to(DEV))[0].double().cpu()
    # p is 1 / 101, off by its exponent's rounding (8 u of 80 log2 e), and rounded to the type
    half, own = rows64.steps(dtype)[0], dout.double().view(Hk, H // Hk, D)
    want, mag = own.sum(1) / n, own.abs().sum(1) / n
    close(dv[at], (want.expand(n, Hk, D), (mag * (half + 8 * 120 * 2.0 ** -24)).expand(n, Hk, D)), dtype, "dv")
    # the others' weight is e^-80 = 1.8e-35 of that, which fp32 and bf16 still hold: two
    # roundings of 2^-8 and the exponent's
    rest = 1.02 * (1 + 2 * 2.0 ** -8) * float(torch.exp(torch.tensor(-80.0, dtype=torch.float64))) * mag
    assert bool((dv[1:at[1]].abs() <= rest).all())


@pytest.mark.parametrize("far", ["keys", "rows"])
def test_gradients_of_the_last_segment(far):
    """The last of two segments, behind 2^32 elements of k, v, dk and dv, or of q, dout,
    out and dq: its rows, keys and gradients against 64 bits, one head alone."""
    n, m, h = 40, 300, 101
    R, K = (ROWS, m + 10) if far == "rows" else (n + 3, ROWS)
    g = rng(R, K)
    q, k, v, dout = (torch.zeros(rows, HEADS, WIDTH, dtype=BF16, device=DEV) for rows in (R, K, K, R))
    ends = [normal(g, rows, HEADS, WIDTH, dtype=BF16) for rows in (n, m, m, n)]
    for t, end in zip((q, k, v, dout), ends):
        t[-end.shape[0]:] = end.to(DEV)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    out = G.segment_attention(*leaves, torch.tensor([0, R - n, R], device=DEV), torch.tensor([0, K - m, K], device=DEV),
                              causal=True)
    grads = torch.autograd.grad(out, leaves, dout)
    one = [t[:, h:h + 1] for t in ends]
    want = rows64.attention(*one[:3], [0, n], [0, m], True, WIDTH ** -0.5, one[3])
    for name, t, w, rows in zip(("out", "dq", "dk", "dv"), (out, *grads), want, (n, n, m, m)):
        close(t[-rows:, h:h + 1], w, BF16, name)
        bound = w[1] + half_step(w[0].abs() + w[1], BF16)
        reach = float((w[0].abs() / bound).max())
        log(f"{far} {name}: bound 1 / {reach:.3g} of the largest value")
        # zeros, or another segment's rows, would be off by more than five bounds.  (A sum of n
        # like terms of either sign is about 1 / sqrt(n) of their magnitudes, its largest
        # element among thousands 3 to 4 times that, the bound 2^-8 of them: 256 * 3.5 / sqrt(300)
        # is 50 for one rounding a term, and dq's terms are rounded or off three times as much.)
        assert reach > 5
        # nothing of it is written into the segment ahead, whose gradients are zero
        assert not bool(t[:-rows][-5000:].any()) and not bool(t[:3].any())


def test_loss_of_rows_past_2_31_bytes():
    """x of just over 2 GiB, a few rows with a class, the last ones among them: what
    the other rows hold (NaN) reaches nothing."""
    R, I, V = 524289 + 300, 2048, 40
    x = torch.full((R, I), float("nan"), dtype=BF16, device=DEV)
    assert x.numel() * 2 > 2 ** 31
    at = torch.tensor([0, 1, 262143, 262144, 262145, 500000, 524287, 524288, 524289, R - 2, R - 1])
    g = rng(R)
    rows, w = normal(g, at.numel(), I, dtype=BF16), normal(g, V, I, dtype=BF16, scale=2 * I ** -0.5)
    target = torch.full((R,), -1)
    target[at] = torch.randint(0, V, (at.numel(),), generator=g)
    x[at.to(DEV)] = rows.to(DEV)
    leaves = [x.requires_grad_(), w.to(DEV).requires_grad_()]
    dloss = torch.zeros(R)
    dloss[at] = normal(g, at.numel())
    loss = G.linear_cross_entropy(*leaves, target.to(DEV), "none")
    dx, dw = torch.autograd.grad(loss, leaves, dloss.to(DEV))
    want = rows64.loss(rows, w, target[at], "none", dloss[at])
    close(loss.detach()[at.to(DEV)], want[0], torch.float32, "loss")
    close(dx[at.to(DEV)], want[1], BF16, "dx")
    close(dw, want[2], BF16, "dw")
    assert int((loss != 0).sum()) == at.numel()
    dx[at.to(DEV)] = 0.0
    assert not bool(dx.any())


def test_classes_past_2_32_elements():
    """A few rows against classes of 2^32 elements and more, zeros but for a few: the
    loss and both gradients in closed form."""
    R, I, V = 3, 256, 2 ** 24 + 77
    g = rng(V)
    w = torch.zeros(V, I, dtype=BF16, device=DEV)
    assert w.numel() > 2 ** 32
    at = torch.tensor([5, 2 ** 23 - 1, 2 ** 23 + 3, 2 ** 24 - 1, 2 ** 24, V - 1])
    few, x = normal(g, at.numel(), I, dtype=BF16, scale=2 * I ** -0.5), normal(g, R, I, dtype=BF16, scale=3.0)
    few[3:] += 0.02 * x.sign()                         # logits of about 12: a share of the weight next to e^16.6
    w[at.to(DEV)] = few.to(DEV)
    target = at[torch.tensor([5, 1, 4])]
    leaves = [x.to(DEV).requires_grad_(), w.requires_grad_()]
    loss = G.linear_cross_entropy(*leaves, target.to(DEV), "none")
    dx, dw = torch.autograd.grad(loss, leaves, torch.ones(R, device=DEV))
    xd, fd = x.double(), few.double()
    logits = xd @ fd.T
    others = torch.log(torch.full((R, 1), float(V - at.numel()), dtype=torch.float64))
    lse = torch.logsumexp(torch.cat([logits, others], 1), 1)
    own = logits[torch.arange(R), torch.tensor([5, 1, 4])]
    u = 2.0 ** -24
    mag = xd.abs() @ fd.abs().T
    # logits off by 2 I u of their magnitudes, sums of the tiles' like terms, 32 of them at a time
    each = 2 * I * u * float(mag.max()) + 8 * 40 * u + (128 + 2 * V / 128 / 32) * u
    assert bool(((loss.detach().double().cpu() - (lse - own)).abs() <= each + 4 * u * lse).all())
    p = torch.exp(logits - lse[:, None])
    d = p.clone()
    d[torch.arange(R), torch.tensor([5, 1, 4])] -= 1
    half = 2.0 ** -8                                   # bf16: d once, the output once
    size = (d.abs() * (half + 2 * each + 8 * u) + p * 2 * each) @ fd.abs()
    want = d @ fd
    assert bool(((dx.detach().double().cpu() - want).abs() <= 1.02 * (size + half * (want.abs() + size))).all())
    want = d.T @ xd
    size = (d.abs() * (half + 2 * each + 8 * u) + p * 2 * each).T @ xd.abs()
    got = dw[at.to(DEV)].double().cpu()
    assert bool(((got - want).abs() <= 1.02 * (size + half * (want.abs() + size))).all())
    assert float((want.abs() / (size + half * want.abs())).max()) > 20
    # every other class has p = exp(-lse)
    rest = torch.exp(-lse) @ xd
    tol = torch.exp(-lse) @ xd.abs() * (2 * half + 3 * each)
    for a in (6, 2 ** 23, 2 ** 24 - 2, 2 ** 24 + 1, V - 2):
        assert bool(((dw[a].double().cpu() - rest).abs() <= 1.02 * (tol + half * rest.abs())).all())
