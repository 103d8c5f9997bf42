"""The loss of a linear classifier against its plain form in 64 bits
(tests/rows64.py, which derives the tolerances)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_attention import SLACK, close  # noqa: E402
from tests.test_gpu_rows import TYPES, guarded, half_step, normal, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log


def case(R, I, V, dtype, drop=0.2, seed=0):
    """x, w and targets, some rows without a class: NaN stands in them."""
    g = rng(R, I, V, seed)
    x, w = normal(g, R, I, dtype=dtype), normal(g, V, I, dtype=dtype, scale=2 * I ** -0.5)
    target = torch.randint(0, V, (R,), generator=g)
    gone = torch.rand(R, generator=g) < drop
    far = torch.tensor([-1, V, -100, 2 ** 40, -2 ** 40])[torch.randint(0, 5, (R,), generator=g)]
    target = torch.where(gone, far, target)
    x[gone] = float("nan")
    return x, w, target


def on_gpu(x, w, target, reduction, dloss):
    leaves = [x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()]
    loss = G.linear_cross_entropy(*leaves, target.to(DEV), reduction)
    assert loss.dtype == torch.float32 and loss.shape == dloss.shape
    return [loss, *torch.autograd.grad(loss, leaves, dloss.to(DEV))]


def compare(R, I, V, kind, reduction, drop=0.2):
    log(f"loss R={R} I={I} V={V} {kind} {reduction} drop={drop}")
    dtype = TYPES[kind]
    x, w, target = case(R, I, V, dtype, drop)
    dloss = normal(rng(7, R), R if reduction == "none" else 1).view((R,) if reduction == "none" else ())
    got = on_gpu(x, w, target, reduction, dloss)
    want = rows64.loss(x, w, target, reduction, dloss)
    close(got[0], want[0], torch.float32, "loss")
    close(got[1], want[1], dtype, "dx")
    close(got[2], want[2], dtype, "dw")
    gone = (target < 0) | (target >= V)
    assert not bool(got[1].detach().cpu()[gone].any())
    if reduction == "none":
        assert not bool(got[0].detach().cpu()[gone].any())
    with torch.no_grad():
        assert torch.equal(G.linear_cross_entropy(x.to(DEV), w.to(DEV), target.to(DEV), reduction), got[0].detach())


SIZES = [(1, 1, 1), (1, 8, 2), (2, 3, 5), (31, 16, 33), (33, 40, 63), (64, 64, 64), (65, 32, 65), (128, 24, 127), (129, 72, 128),
         (130, 65, 129), (200, 128, 47), (257, 33, 300), (300, 7, 1000), (700, 100, 3), (2049, 20, 17), (5000, 48, 90)]


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,I,V", SIZES)
def test_sizes(R, I, V, kind, reduction):
    compare(R, I, V, kind, reduction)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,I,V", [(600, 136, 33000), (70, 50, 20011), (8200, 130, 2100), (40000, 8, 40)])
def test_parts_and_large_tiles(R, I, V, kind):
    """dx in parts of the classes, dw in chunks of rows, 256 x 256 tiles, rows moved
    to whole 16 bytes."""
    compare(R, I, V, kind, "mean", 0.1)


@pytest.mark.parametrize("R,I,V", [(2061, 2048, 4099), (2048, 2048, 4096)])
def test_long_fp32_sums(R, I, V):
    """dx in two parts of the classes and dw over all rows at once, each longer than
    a run of 2,048 that is summed in one chain, or as long."""
    compare(R, I, V, "fp32", "mean", 0.0)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("drop", [0.0, 1.0, 0.97])
def test_all_no_and_few_rows_with_a_class(drop, kind):
    compare(400, 64, 50, kind, "none", drop)
    compare(400, 64, 200, kind, "mean", drop)
    compare(3000, 24, 40, kind, "sum", drop)


def test_no_rows():
    x, w = torch.empty(0, 16, device=DEV, requires_grad=True), torch.ones(5, 16, device=DEV, requires_grad=True)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    for reduction in ("none", "sum", "mean"):
        loss = G.linear_cross_entropy(x, w, t, reduction)
        dx, dw = torch.autograd.grad(loss, [x, w], torch.ones_like(loss))
        assert dx.shape == (0, 16) and not bool(dw.any()) and loss.numel() == (0 if reduction == "none" else 1)
        assert reduction == "none" or float(loss) == 0.0


def test_pieces_of_the_classes():
    """More classes than the gradient of the logits is held for at a time: 1,100,000
    rows of 16-bit values leave 256 at once.  Each row's loss and dx, and dw, by
    torch in 64 bits on the GPU, whose own rounding is nothing beside the bounds:
    loss 2^-24 * (2 * 2 I mag + 64 terms), gradients two roundings of 2^-9 each on
    terms that add up to at most sum|d||w| and sum|d||x|."""
    R, I, V = 1100000, 16, 600
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(R, I, generator=g, device=DEV).to(torch.bfloat16).requires_grad_()
    w = (torch.randn(V, I, generator=g, device=DEV) * 0.5).to(torch.bfloat16).requires_grad_()
    target = torch.randint(-1, V, (R,), generator=g, device=DEV)
    dloss = torch.rand(R, generator=g, device=DEV)
    loss = G.linear_cross_entropy(x, w, target, "none")
    dx, dw = torch.autograd.grad(loss, [x, w], dloss)
    live = target >= 0
    wd = w.detach().double()
    dw64, dwmag = torch.zeros(V, I, dtype=torch.float64, device=DEV), torch.zeros(V, I, dtype=torch.float64, device=DEV)
    for a in range(0, R, 100000):
        xs, t, on = x.detach()[a:a + 100000].double(), target[a:a + 100000], live[a:a + 100000]
        logits = xs @ wd.t().contiguous()
        lse = torch.logsumexp(logits, 1)
        own = logits.gather(1, t.clamp(min=0)[:, None])[:, 0]
        mag = (xs.abs() @ wd.abs().t().contiguous()).amax(1)
        want = torch.where(on, lse - own, torch.zeros_like(lse))
        tol = 2.0 ** -24 * (4 * 2 * I * mag + 200 + 8 * want.abs())
        assert bool(((loss.detach()[a:a + 100000] - want).abs() <= tol).all())
        d = torch.exp(logits - lse[:, None])
        d[torch.arange(t.numel(), device=DEV), t.clamp(min=0)] -= 1
        d *= (dloss[a:a + 100000].double() * on)[:, None]
        size = d.abs() @ wd.abs()
        assert bool(((dx[a:a + 100000].double() - d @ wd).abs() <= 2.02 * 2.0 ** -9 * size * 2).all())
        dw64 += d.t().contiguous() @ xs
        dwmag += d.abs().t().contiguous() @ xs.abs()
    # 1,100,000 terms to a sum: their additions count 2^-24 each beside the roundings
    assert bool(((dw.double() - dw64).abs() <= (2.02 * 2.0 ** -8 + R / 256 * 2.0 ** -24) * dwmag).all())


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_large_and_lowest_logits(kind):
    """Logits far apart: one class has all the weight, the others none."""
    dtype = TYPES[kind]
    x = torch.full((3, 2), 100.0, dtype=dtype)
    w = torch.zeros(130, 2, dtype=dtype)
    w[7], w[120] = 100.0, -100.0
    target = torch.tensor([7, 120, 0])
    loss, dx, dw = on_gpu(x, w, target, "none", torch.ones(3))
    assert loss.tolist() == [0.0, 40000.0, 20000.0]
    want = torch.tensor([[0.0, 0.0], [200.0, 200.0], [100.0, 100.0]])
    assert torch.equal(dx.cpu().float(), want)
    expect = torch.zeros(130, 2)
    expect[7], expect[120], expect[0] = 200.0, -100.0, -100.0
    assert torch.equal(dw.cpu().float(), expect)


def test_small_gradients_of_fp16_keep_their_bits():
    """A mean's gradient times tiny probabilities: held by its power of two."""
    x, w, target = case(500, 32, 4000, torch.float16, 0.0)
    for scale in (1.0, 2.0 ** -20, 2.0 ** 10):
        dloss = torch.full((500,), scale)
        got = on_gpu(x, w, target, "none", dloss)
        want = rows64.loss(x, w, target, "none", dloss)
        close(got[1], want[1], torch.float16, "dx")
        close(got[2], want[2], torch.float16, "dw")


def test_nan_and_zero_gradients():
    x, w, target = case(40, 16, 30, torch.float32, 0.0)
    dloss = torch.zeros(40)
    _, dx, dw = on_gpu(x, w, target, "none", dloss)
    assert not bool(dx.any()) and not bool(dw.any())
    dloss[5] = float("inf")
    _, dx, dw = on_gpu(x, w, target, "none", dloss)
    assert not bool(torch.isfinite(dx[5]).any()) and bool(torch.isfinite(torch.cat([dx[:5], dx[6:]])).all())
    x[3] = float("nan")                                 # a row with a class keeps its NaN
    loss, dx, dw = on_gpu(x, w, target, "none", torch.ones(40))
    assert bool(torch.isnan(loss[3])) and bool(torch.isfinite(torch.cat([loss[:3], loss[4:]])).all())
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isfinite(torch.cat([dx[:3], dx[4:]])).all())


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_any_alignment_and_guarded_outputs(kind, shift):
    dtype = TYPES[kind]
    x, w, target = case(140, 64, 70, dtype)

    def at(t):
        whole = torch.zeros(t.numel() + shift + 40, dtype=dtype, device=DEV)
        whole[shift:shift + t.numel()] = t.reshape(-1).to(DEV)
        return whole[shift:shift + t.numel()].view(t.shape)

    xa, wa, ta = at(x), at(w), target.to(DEV)
    loss, a = guarded((140,), torch.float32)
    dx, b = guarded((140, 64), dtype)
    dw, c = guarded((70, 64), dtype)
    dloss = normal(rng(9), 140)
    state = G.spmm_linear_cross_entropy(xa, wa, ta, loss, "none")
    G.spmm_linear_cross_entropy_backward(xa, wa, ta, dloss.to(DEV), dx, dw, state, "none")
    want = rows64.loss(x, w, target, "none", dloss)
    close(loss, want[0], torch.float32, "loss")
    close(dx, want[1], dtype, "dx")
    close(dw, want[2], dtype, "dw")
    a(), b(), c()
    only, d = guarded((70, 64), dtype)
    G.spmm_linear_cross_entropy_backward(xa, wa, ta, dloss.to(DEV), None, only, state, "none")
    assert torch.equal(only, dw)
    only2, e = guarded((140, 64), dtype)
    G.spmm_linear_cross_entropy_backward(xa, wa, ta, dloss.to(DEV), only2, None, state, "none")
    assert torch.equal(only2, dx)
    d(), e()


def test_strided_and_broadcast_inputs():
    g = rng(14)
    wide, target = normal(g, 60, 48).to(DEV), torch.randint(0, 20, (60,), generator=g).to(DEV)
    w = normal(g, 40, 24).to(DEV)
    x = wide[:, ::2].requires_grad_()
    packed = x.detach().contiguous().requires_grad_()
    a, b = G.linear_cross_entropy(x, w[::2], target), G.linear_cross_entropy(packed, w[::2].contiguous(), target)
    assert torch.equal(a, b)
    assert torch.equal(torch.autograd.grad(a, x)[0], torch.autograd.grad(b, packed)[0])
    one = normal(g, 1, 24).to(DEV).requires_grad_()
    loss = G.linear_cross_entropy(one.expand(60, 24), w, target, "sum")
    assert torch.autograd.grad(loss, one)[0].shape == one.shape


def test_two_runs_give_the_same_bits():
    x, w, target = case(3000, 72, 5000, torch.bfloat16)
    runs = [on_gpu(x, w, target, "mean", torch.ones(())) for _ in range(2)]
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_gradients_against_differences():
    """As for the attention: the slope of the kernels' own loss, what the
    difference leaves out taken from 64 bits, the rest within rounding over 2 h."""
    x, w, target = case(150, 20, 45, torch.float32, 0.0)
    h, one = 2.0 ** -5, torch.ones(())
    grads = on_gpu(x, w, target, "sum", one)[1:]
    exact = rows64.loss(x, w, target, "sum", one)[1:]
    g = rng(98)
    for i in range(2):
        p = [x, w]
        ends = [p[i] + h * s * (v := normal(g, *p[i].shape) if s > 0 else v) for s in (1, -1)]
        moved = (ends[0].double() - ends[1].double()) / (2 * h)
        f, f64, err = [], [], 0.0
        for e in ends:
            at = [e if j == i else t for j, t in enumerate(p)]
            f.append(float(G.linear_cross_entropy(at[0].to(DEV), at[1].to(DEV), target.to(DEV), "sum")))
            value, bound = rows64.loss(*at, target, "sum")[0]
            f64.append(float(value))
            err += float(bound + half_step(value.abs() + bound, torch.float32))
        value, bound = exact[i]
        left_out = (f64[0] - f64[1]) / (2 * h) - float((value * moved).sum())
        slope = float((grads[i].double().cpu() * moved).sum())
        tol = SLACK * (err / (2 * h) + float((moved.abs() * (bound + half_step(value.abs() + bound, torch.float32))).sum()))
        assert abs(slope + left_out - (f[0] - f[1]) / (2 * h)) <= tol
