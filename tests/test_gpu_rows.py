"""Row operators (route, dispatch, combine, segment product, layer norm)
against plain implementations in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32.  A sum of n fp32 terms in any
order, one rounding per term, is off by at most n * u * sum|terms| (first
order; a factor 1.01 covers the rest at these sizes); where the order is a
tree, n is its longest chain.  An output of type t is rounded once more: half
a step, finfo(t).eps / 2 of the value, and half the smallest subnormal.  The
matrix cores may truncate where they add, so a product's terms count a whole
step, 2 u, each.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24
SLACK = 1.01


def half_step(ref, dtype):
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def close(got, ref, before, dtype, what):
    """|got - ref| <= before (the error ahead of the last rounding) + half a
    step of the value that was rounded."""
    err = (got.double().cpu() - ref).abs()
    tol = SLACK * (before + half_step(ref.abs() + before, dtype))
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error {float(err.max()):.3e}, "
                           f"worst ratio {float((err / tol.clamp(min=1e-300)).max()):.3g}")


def rng(*key):
    g = torch.Generator()
    g.manual_seed(sum((i + 1) * 7919 * int(k) for i, k in enumerate(key)) + 5)
    return g


def normal(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype)


def guarded(shape, dtype, fill=-3.0, pad=24):
    """A tensor of `shape` inside a longer array, and a check that the array's
    elements around it kept their value."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=DEV)

    def untouched():
        edge = torch.cat([whole[:pad], whole[pad + n:]])
        assert bool((edge == fill).all()), "elements around the output were written"
    return whole[pad:pad + n].view(shape), untouched


def pairs_of(g, T, k, E, kind):
    if kind == "one":
        e = torch.full((T, k), E - 1)
    elif kind == "none":
        e = torch.full((T, k), -1)
    else:
        e = torch.randint(0, E, (T, k), generator=g)
        if kind == "some":
            gone = torch.rand(T, k, generator=g) < 0.3
            far = torch.tensor([-1, E, -2 ** 40, 2 ** 40])[torch.randint(0, 4, (T, k), generator=g)]
            e = torch.where(gone, far, e)
    return e.to(torch.int64)


def plain_route(e, E):
    key = e.reshape(-1).numpy()
    key = np.where((key < 0) | (key >= E), E, key)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    return np.searchsorted(key[order], np.arange(E + 1)), order, position.reshape(e.shape)


# --------------------------------------------------------------------- route

@pytest.mark.parametrize("T,k,E,kind", [
    (0, 2, 4, "all"), (0, 1, 2048, "all"), (1, 1, 1, "all"), (1, 3, 2, "some"), (63, 1, 8, "all"), (64, 2, 8, "all"),
    (65, 2, 511, "some"), (512, 2, 511, "all"), (513, 2, 7, "some"), (1024, 4, 64, "one"), (1365, 3, 64, "some"),
    (4096, 1, 511, "some"), (4097, 1, 100, "all"), (2048, 8, 16, "none"), (16384, 1, 511, "some"), (16385, 1, 511, "some"),
    (300, 2, 512, "all"), (5000, 2, 2048, "some"), (40000, 3, 33, "some"), (70001, 8, 255, "all"),
    (300007, 2, 3, "one"), (1100000, 4, 129, "some"),
    (262144, 2, 64, "one"), (131073, 4, 1024, "some"), (131073, 4, 1025, "some"), (600001, 1, 200, "none")])
def test_route(T, k, E, kind):
    log(f"route T={T} k={k} E={E} {kind}")
    e = pairs_of(rng(T, k, E), T, k, E, kind)
    want = plain_route(e, E)
    for _ in range(2):
        r = G.RowRoute(e.to(DEV), E)
        assert np.array_equal(r.offsets.cpu().numpy(), want[0])
        assert np.array_equal(r.order.cpu().numpy(), want[1])
        assert np.array_equal(r.position.cpu().numpy(), want[2])


def test_route_of_one_expert_per_row_and_of_a_view():
    e = pairs_of(rng(4), 777, 1, 9, "some")[:, 0]
    r = G.RowRoute(e.to(DEV), 9)
    assert r.position.shape == (777, 1)
    assert np.array_equal(r.order.cpu().numpy(), plain_route(e, 9)[1])
    wide = pairs_of(rng(5), 50, 6, 9, "some")
    r = G.RowRoute(wide.to(DEV)[:, ::2], 9)          # a strided view is taken as its values
    assert np.array_equal(r.position.cpu().numpy(), plain_route(wide[:, ::2], 9)[2])


def test_route_writes_inside_its_arrays():
    e = pairs_of(rng(6), 333, 3, 40, "some").to(DEV)
    offsets, a = guarded((41,), torch.int64, -3)
    order, b = guarded((999,), torch.int32, -3)
    position, c = guarded((333, 3), torch.int32, -3)
    G.spmm_route_build(e, 40, offsets, order, position)
    want = plain_route(e.cpu(), 40)
    assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(order.cpu().numpy(), want[1])
    a(), b(), c()


# ------------------------------------------------------------------ exchange

EXCHANGE = [(1, 1, 1, 1, "all"), (5, 2, 3, 3, "some"), (64, 4, 8, 64, "all"), (33, 3, 5, 7, "some"),
            (129, 2, 16, 129, "some"), (50, 9, 20, 40, "some"), (200, 1, 6, 1433, "some"), (17, 2, 4, 4099, "all"),
            (40, 2, 3, 16, "none"), (700, 5, 600, 2, "some"), (3, 70, 9, 24, "some")]


@pytest.mark.parametrize("weights", ["none", "fp32", "own"])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("T,k,E,N,which", EXCHANGE)
def test_exchange(T, k, E, N, which, kind, weights):
    log(f"exchange T={T} k={k} E={E} N={N} {which} {kind} weights={weights}")
    dtype, g = TYPES[kind], rng(T, k, E, N)
    e = pairs_of(g, T, k, E, which)
    offsets, order, position = plain_route(e, E)
    kept = int(offsets[-1])
    position = torch.from_numpy(position)
    there = position < kept
    x, rows = normal(g, T, N, dtype=dtype), normal(g, T * k, N, dtype=dtype)
    rows[kept:] = float("nan")                       # rows of no expert are not read
    dxs, dout = normal(g, T * k, N, dtype=dtype), normal(g, T, N, dtype=dtype)
    dxs[kept:] = float("inf")
    w = None if weights == "none" else torch.rand(T, k, generator=g).to(torch.float32 if weights == "fp32" else dtype)
    r = G.RowRoute(e.to(DEV), E)
    xd, rd = x.to(DEV).requires_grad_(), rows.to(DEV).requires_grad_()
    wd = None if w is None else w.to(DEV).requires_grad_()

    xs = G.dispatch(r, xd)
    want = torch.zeros(T * k, N, dtype=dtype)
    want[position[there]] = x[torch.arange(T)[:, None].expand(T, k)[there]]
    assert torch.equal(xs.detach().cpu(), want)
    dx, = torch.autograd.grad(xs, xd, dxs.to(DEV))
    zero = torch.zeros((), dtype=torch.float64)
    d = torch.where(there[:, :, None], dxs.double()[position], zero)
    close(dx, d.sum(1), k * U * d.abs().sum(1), dtype, "dx")

    out = G.combine(r, rd, wd)
    w64 = torch.ones(T, k, dtype=torch.float64) if w is None else w.double()
    y = torch.where(there[:, :, None], rows.double()[position], zero)
    terms = w64[:, :, None] * y
    close(out.detach(), terms.sum(1), k * U * terms.abs().sum(1), dtype, "out")
    grads = torch.autograd.grad(out, [rd] + ([] if w is None else [wd]), dout.to(DEV))
    drows = torch.zeros(T * k, N, dtype=torch.float64)
    drows[position[there]] = (w64[:, :, None] * dout.double()[:, None, :])[there]
    close(grads[0], drows, U * drows.abs(), dtype, "drows")
    if w is not None:
        dots = y * dout.double()[:, None, :]
        close(grads[1], dots.sum(2), N * U * dots.abs().sum(2), w.dtype, "dweight")
        assert bool((grads[1].cpu()[~there] == 0).all())


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_exchange_writes_inside_its_arrays(kind):
    dtype, g = TYPES[kind], rng(31)
    T, k, E, N = 37, 3, 5, 45
    e = pairs_of(g, T, k, E, "some").to(DEV)
    r = G.RowRoute(e, E)
    x, w = normal(g, T, N, dtype=dtype).to(DEV), torch.rand(T, k, generator=g).to(DEV)
    rows, dout = normal(g, T * k, N, dtype=dtype).to(DEV), normal(g, T, N, dtype=dtype).to(DEV)
    xs, a = guarded((T * k, N), dtype)
    out, b = guarded((T, N), dtype)
    drows, c = guarded((T * k, N), dtype)
    dw, d = guarded((T, k), torch.float32)
    G.spmm_route_dispatch(r, x, xs)
    G.spmm_route_combine(r, rows, w, out)
    G.spmm_route_combine_backward(r, rows, w, dout, drows, dw)
    a(), b(), c(), d()
    assert torch.equal(xs, G.dispatch(r, x)) and torch.equal(out, G.combine(r, rows, w))
    # each gradient alone gives the same bits, and so does the weighted dispatch
    only_rows, only_w, again = torch.empty_like(rows), torch.empty_like(w), torch.empty_like(rows)
    G.spmm_route_combine_backward(r, None, w, dout, only_rows, None)
    G.spmm_route_combine_backward(r, rows, w, dout, None, only_w)
    G.spmm_route_dispatch(r, dout, again, w)
    assert torch.equal(only_rows, drows) and torch.equal(only_w, dw) and torch.equal(again, drows)


@pytest.mark.parametrize("T,k,N,kind", [(720000, 3, 2048, "bf16"), (50021, 3, 1433, "fp16"), (300007, 2, 64, "fp32"),
                                        (700001, 2, 100, "fp16")])
def test_exchange_of_large_calls(T, k, N, kind):
    """Calls that stream past the cache, and (2048 wide) offsets past 2^32
    elements; rows at the ends and around the borders, and random ones."""
    dtype, g, E = TYPES[kind], rng(T, N), 9
    e = pairs_of(g, T, k, E, "some")
    r = G.RowRoute(e.to(DEV), E)
    order, kept = r.order.cpu().long(), int(r.offsets[-1])
    position = r.position.cpu().long()
    x = torch.randn(T, N, device=DEV, dtype=dtype)
    xs = G.dispatch(r, x)
    at = torch.cat([torch.randint(0, T * k, (3000,), generator=g),
                    torch.tensor([0, 1, kept - 1, kept, T * k - 1, T * k // 2])]
                   + [torch.arange(min(T * k, c) - 2, min(T * k, c + 3)) for c in (2 ** 31 // N, 2 ** 32 // N)])
    want = torch.where((at < kept)[:, None], x[(order[at] // k).to(DEV)].cpu(), torch.zeros((), dtype=dtype))
    assert torch.equal(xs[at.to(DEV)].cpu(), want)
    w = torch.rand(T, k, generator=g)
    wd = w.to(DEV)
    out, drows, dw = torch.empty_like(x), torch.empty_like(xs), torch.empty_like(wd)
    G.spmm_route_combine(r, xs, wd, out)
    t = torch.cat([torch.randint(0, T, (1500,), generator=g), torch.tensor([0, T - 1])])
    there = position[t] < kept
    rows = torch.where(there[:, :, None], xs[position[t].to(DEV)].double().cpu(), torch.zeros((), dtype=torch.float64))
    terms = w[t].double()[:, :, None] * rows
    close(out[t.to(DEV)], terms.sum(1), k * U * terms.abs().sum(1), dtype, "out")
    G.spmm_route_combine_backward(r, xs, wd, x, drows, dw)
    d = x[(order[at] // k).to(DEV)].double().cpu()
    grad = torch.where((at < kept)[:, None], w.reshape(-1)[order[at]].double()[:, None] * d, torch.zeros((), dtype=torch.float64))
    close(drows[at.to(DEV)], grad, U * grad.abs(), dtype, "drows")
    dots = rows * x[t.to(DEV)].double().cpu()[:, None, :]
    close(dw[t.to(DEV)], dots.sum(2), N * U * dots.abs().sum(2), torch.float32, "dweight")


def test_infinite_weights_and_rows_follow_the_formula():
    e = torch.tensor([[0, 1], [1, -1], [-1, -1]], device=DEV)
    r = G.RowRoute(e, 2)
    rows = torch.ones(6, 4, device=DEV)
    rows[int(r.position[0, 1])] = float("inf")
    w = torch.tensor([[0.0, 1.0], [2.0, float("nan")], [float("inf"), float("nan")]], device=DEV)
    out = G.combine(r, rows, w)
    assert bool(torch.isinf(out[0]).all())
    assert torch.equal(out[1:].cpu(), torch.tensor([[2.0] * 4, [0.0] * 4]))


# ----------------------------------------------------------- segment product

def bounds_of(g, R, E, head, tail):
    cut = torch.sort(torch.randint(head, max(head, R - tail) + 1, (E - 1,), generator=g)).values
    return torch.cat([torch.tensor([head]), cut, torch.tensor([max(head, R - tail)])]).to(torch.int64)


SEGMENT = [(0, 3, 8, 8, 0, 0), (1, 1, 1, 1, 0, 0), (5, 3, 7, 9, 1, 1), (40, 4, 16, 8, 0, 0), (300, 4, 64, 128, 0, 0),
           (129, 2, 130, 70, 0, 3), (1000, 70, 33, 65, 5, 140), (257, 3, 200, 136, 130, 0), (64, 150, 24, 40, 0, 0),
           (777, 1, 129, 257, 0, 0), (4000, 2, 48, 33, 0, 100), (9, 5, 520, 264, 0, 0), (640, 3, 256, 128, 0, 0),
           (2000, 5, 1, 3, 0, 0)]


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,E,I,O,head,tail", SEGMENT)
def test_segment_matmul(R, E, I, O, head, tail, kind):
    log(f"segment R={R} E={E} I={I} O={O} head={head} tail={tail} {kind}")
    dtype, g = TYPES[kind], rng(R, E, I, O)
    b = bounds_of(g, R, E, min(head, R), tail)
    x, w, dy = normal(g, R, I, dtype=dtype), normal(g, E, I, O, dtype=dtype), normal(g, R, O, dtype=dtype)
    inside = torch.zeros(R, dtype=torch.bool)
    inside[int(b[0]):int(b[-1])] = True
    x[~inside] = float("nan")                        # rows outside the segments do not enter
    dy[~inside] = float("inf")
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = G.segment_matmul(xd, wd, b.to(DEV))
    dx, dw = torch.autograd.grad(y, [xd, wd], dy.to(DEV))
    for e in range(E):
        s = slice(int(b[e]), int(b[e + 1]))
        X, W, D = x[s].double(), w[e].double(), dy[s].double()
        close(y.detach()[s], X @ W, 2 * U * I * (X.abs() @ W.abs()), dtype, f"y of segment {e}")
        close(dx[s], D @ W.t(), 2 * U * O * (D.abs() @ W.abs().t()), dtype, f"dx of segment {e}")
        n = max(1, X.shape[0])
        close(dw[e], X.t() @ D, 2 * U * n * (X.abs().t() @ D.abs()), dtype, f"dw of segment {e}")
    assert bool((y.detach().cpu()[~inside] == 0).all()) and bool((dx.cpu()[~inside] == 0).all())


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("R,E,I,O", [(200, 3, 72, 144), (12, 6, 136, 88)])
def test_segment_product_at_any_alignment(R, E, I, O, shift, kind):
    """Operands that start in the middle of a 16-byte group, outputs inside a
    longer array; the same bits as aligned ones, nothing around them written."""
    dtype, g = TYPES[kind], rng(9, shift)
    b = bounds_of(g, R, E, 0, 7 if R > 100 else 1).to(DEV)

    def moved(t):
        whole = torch.zeros(t.numel() + shift, dtype=dtype, device=DEV)
        whole[shift:] = t.reshape(-1).to(DEV)
        return whole[shift:].view(t.shape)
    x, w, dy = normal(g, R, I, dtype=dtype), normal(g, E, I, O, dtype=dtype), normal(g, R, O, dtype=dtype)
    outs = []
    for m in (moved, lambda t: t.to(DEV)):
        y, c1 = guarded((R, O), dtype, pad=24 + shift)
        dx, c2 = guarded((R, I), dtype, pad=24 + shift)
        dw, c3 = guarded((E, I, O), dtype, pad=24 + shift)
        G.spmm_segment_product(m(x), m(w), b, y)
        G.spmm_segment_product_dx(m(dy), m(w), b, dx)
        G.spmm_segment_product_dw(m(x), m(dy), b, dw)
        c1(), c2(), c3()
        outs.append((y.clone(), dx.clone(), dw.clone()))
    for p, q in zip(*outs):
        assert torch.equal(p, q)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_segment_rows_of_another_segment_do_not_leak(kind):
    """NaN rows and NaN weights of one segment stay in its own outputs."""
    dtype, g = TYPES[kind], rng(12)
    b = torch.tensor([0, 70, 70, 135, 200], device=DEV)
    x, w, dy = (normal(g, *s, dtype=dtype).to(DEV) for s in ((200, 72), (4, 72, 40), (200, 40)))
    clean = [t.clone() for t in (x, w, dy)]
    x[70:135], w[1:3], dy[70:135] = float("nan"), float("inf"), float("nan")

    def products(x, w, dy):
        y, dx, dw = x.new_empty(200, 40), x.new_empty(200, 72), torch.empty_like(w)
        G.spmm_segment_product(x, w, b, y)
        G.spmm_segment_product_dx(dy, w, b, dx)
        G.spmm_segment_product_dw(x, dy, b, dw)
        return y, dx, dw
    got, want = products(x, w, dy), products(*clean)
    other = torch.ones(200, dtype=torch.bool, device=DEV)
    other[70:135] = False
    assert torch.equal(got[0][other], want[0][other]) and torch.equal(got[1][other], want[1][other])
    assert torch.equal(got[2][[0, 1, 3]], want[2][[0, 1, 3]]) and bool(torch.isnan(got[0][70:135]).all())


@pytest.mark.parametrize("offsets", [[0, 6000, 0, 6000, 0, 6000], [6000, 0, 0, 0, 0, 0], [-5, 2 ** 40, 3, -2 ** 40, 6000, 1]])
@pytest.mark.parametrize("I,O", [(64, 64), (65, 33)])
def test_segment_offsets_out_of_order_touch_nothing_outside(I, O, offsets):
    """What comes out is not specified; what stands around the outputs stays."""
    R, E = 6000, 5
    x, w, dy = (torch.ones(*s, device=DEV) for s in ((R, I), (E, I, O), (R, O)))
    b = torch.tensor(offsets, device=DEV)
    y, c1 = guarded((R, O), torch.float32)
    dx, c2 = guarded((R, I), torch.float32)
    dw, c3 = guarded((E, I, O), torch.float32)
    G.spmm_segment_product(x, w, b, y)
    G.spmm_segment_product_dx(dy, w, b, dx)
    G.spmm_segment_product_dw(x, dy, b, dw)
    torch.cuda.synchronize()
    c1(), c2(), c3()


def test_segment_products_of_many_rows():
    """Long segments: dw in chunks of rows, more chunks than one scan covers,
    and products whose element offsets pass 2^31."""
    g = rng(41)
    b = torch.tensor([0, 17, 17, 50000, 299000, 300000], device=DEV)
    x, dy = normal(g, 300011, 24).to(DEV), normal(g, 300011, 40).to(DEV)
    dw = torch.empty(5, 24, 40, device=DEV)
    G.spmm_segment_product_dw(x, dy, b, dw)
    for e in range(5):
        X, D = (t[int(b[e]):int(b[e + 1])].double().cpu() for t in (x, dy))
        close(dw[e], X.t() @ D, 2 * U * max(1, len(X)) * (X.abs().t() @ D.abs()), torch.float32, f"dw of segment {e}")
    R, I, O = 1100000, 2048, 16
    x = torch.randn(R, I, device=DEV, dtype=torch.bfloat16)
    w = normal(g, 2, I, O, dtype=torch.bfloat16).to(DEV)
    b = torch.tensor([0, 3, R], device=DEV)
    y = torch.empty(R, O, device=DEV, dtype=torch.bfloat16)
    G.spmm_segment_product(x, w, b, y)
    rows = torch.tensor([0, 3, 524288, 1048575, 1048576, R - 1])
    X, W = x[rows.to(DEV)].double().cpu(), w.double().cpu()
    want = torch.stack([X[i] @ W[0 if r < 3 else 1] for i, r in enumerate(rows.tolist())])
    size = torch.stack([X[i].abs() @ W[0 if r < 3 else 1].abs() for i, r in enumerate(rows.tolist())])
    close(y[rows.to(DEV)], want, 2 * U * I * size, torch.bfloat16, "y far into x")
    dx = torch.empty_like(x)
    G.spmm_segment_product_dx(y, w, b, dx)
    Y = y[rows.to(DEV)].double().cpu()
    want = torch.stack([W[0 if r < 3 else 1] @ Y[i] for i, r in enumerate(rows.tolist())])
    size = torch.stack([W[0 if r < 3 else 1].abs() @ Y[i].abs() for i, r in enumerate(rows.tolist())])
    close(dx[rows.to(DEV)], want, 2 * U * O * size, torch.bfloat16, "dx far into x")


# ---------------------------------------------------------------- layer norm

NORM = [(0, 8), (1, 1), (3, 5), (7, 32), (33, 100), (700, 64), (5000, 16), (5, 1433), (9, 4096), (3, 2056), (2, 8200),
        (3, 20000), (2, 70001), (300, 520)]


@pytest.mark.parametrize("weights", ["none", "fp32", "own"])
@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("R,N", NORM)
def test_layer_norm(R, N, kind, weights):
    log(f"norm R={R} N={N} {kind} weights={weights}")
    dtype, g, eps = TYPES[kind], rng(R, N), 1e-5
    x, dy = normal(g, R, N, dtype=dtype, scale=2.0, shift=0.5), normal(g, R, N, dtype=dtype)
    if R > 2:
        x[1] = 7.0                                   # a row without variance
    wtype = torch.float32 if weights == "fp32" else dtype
    w, b = (None, None) if weights == "none" else (normal(g, N, dtype=wtype), normal(g, N, dtype=wtype))
    xd = x.to(DEV).requires_grad_()
    leaves = [xd] + ([] if w is None else [w.to(DEV).requires_grad_(), b.to(DEV).requires_grad_()])
    y = G.layer_norm(xd, *leaves[1:], eps=eps)
    grads = torch.autograd.grad(y, leaves, dy.to(DEV))

    X, D = x.double(), dy.double()
    W, B = (1.0, 0.0) if w is None else (w.double(), b.double())
    mean = X.mean(1, keepdim=True)
    d = X - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    unit = d * rstd
    chain = 64 + N / 1024                            # longest chain of additions over a row
    e_mean = (chain + 2) * U * X.abs().mean(1, keepdim=True)
    e_d = e_mean + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d * e_d).mean(1, keepdim=True) + (chain + 3) * U * var
    e_rstd = e_var / (2 * (var + eps)) + 6 * U       # relative; eps, the sum, root and division: a step each
    # a relative error a of var + eps moves 1 / sqrt by at most a / 2 * (1 - a) ** -1.5
    a = (e_var / (var + eps)).clamp(max=0.5)
    e_rstd = e_rstd * (1 - a) ** -1.5
    e_unit = e_d * rstd * (1 + e_rstd) + unit.abs() * (e_rstd + 2 * U)
    Wa = 1.0 if w is None else W.abs()
    ref = unit * W + B
    close(y.detach(), ref, Wa * e_unit + 2 * U * (Wa * unit.abs() + ref.abs()), dtype, "y")

    gr = D * W
    mg, mgu = gr.mean(1, keepdim=True), (gr * unit).mean(1, keepdim=True)
    e_mg = (chain + 3) * U * gr.abs().mean(1, keepdim=True)
    e_mgu = (gr.abs() * e_unit).mean(1, keepdim=True) + (chain + 4) * U * (gr * unit).abs().mean(1, keepdim=True)
    parts = gr.abs() + mg.abs() + (unit * mgu).abs()
    inner = gr - mg - unit * mgu
    e_dx = rstd * (1 + e_rstd) * (e_mg + unit.abs() * e_mgu + e_unit * (mgu.abs() + e_mgu) + 5 * U * parts) \
        + rstd * inner.abs() * (e_rstd + U)
    close(grads[0], rstd * inner, e_dx, dtype, "dx")
    if w is not None:
        terms = (D * unit).abs().sum(0)
        close(grads[1], (D * unit).sum(0), (D.abs() * e_unit).sum(0) + (R + 40) * U * terms, wtype, "dweight")
        close(grads[2], D.sum(0), (R + 40) * U * D.abs().sum(0), wtype, "dbias")


@pytest.mark.parametrize("N", [3, 64, 1000, 9000, 70000])
def test_layer_norm_parts_and_bounds(N):
    """Each gradient alone gives the same bits as all of them; nothing outside
    the outputs is written; a weight or a bias alone works."""
    g, R = rng(N), 37
    x, dy, w, b = (normal(g, *s).to(DEV) for s in ((R, N), (R, N), (N,), (N,)))
    y, c0 = guarded((R, N), torch.float32)
    mean, c1 = guarded((R,), torch.float32)
    rstd, c2 = guarded((R,), torch.float32)
    dx, c3 = guarded((R, N), torch.float32)
    dw, c4 = guarded((N,), torch.float32)
    db, c5 = guarded((N,), torch.float32)
    G.spmm_layer_norm(x, w, b, y, mean, rstd)
    G.spmm_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db)
    for c in (c0, c1, c2, c3, c4, c5):
        c()
    assert torch.equal(y, G.layer_norm(x, w, b))
    only = [torch.empty_like(t) for t in (dx, dw, db)]
    G.spmm_layer_norm_backward(dy, x, w, mean, rstd, only[0], None, None)
    G.spmm_layer_norm_backward(dy, x, w, mean, rstd, None, only[1], None)
    G.spmm_layer_norm_backward(dy, x, w, mean, rstd, None, None, only[2])
    assert all(torch.equal(p, q) for p, q in zip(only, (dx, dw, db)))
    assert torch.equal(G.layer_norm(x, w), G.layer_norm(x, w, torch.zeros_like(b)))
    assert torch.equal(G.layer_norm(x, None, b), G.layer_norm(x, torch.ones_like(w), b))


@pytest.mark.parametrize("R,N,kind", [(1100001, 2048, "bf16"), (1100001, 61, "fp32"), (100003, 1433, "fp16")])
def test_layer_norm_of_large_calls(R, N, kind):
    """Calls that stream past the cache and element offsets past 2^31: rows
    against the same rows alone, column sums against 64 bits."""
    dtype = TYPES[kind]
    x, dy = (torch.randn(R, N, device=DEV, dtype=dtype) for _ in range(2))
    w, b = (torch.randn(N, device=DEV) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    G.spmm_layer_norm(x, w, b, y, mean, rstd)
    G.spmm_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db)
    at = torch.cat([torch.randint(0, R, (500,), generator=rng(R)), torch.tensor([0, R - 1, 2 ** 31 // N % R])]).to(DEV)
    few = [t[at].contiguous() for t in (x, dy, mean, rstd)]
    assert torch.equal(y[at], G.layer_norm(few[0], w, b))
    some = torch.empty_like(few[0])
    G.spmm_layer_norm_backward(few[1], few[0], w, few[2], few[3], some, None, None)
    assert torch.equal(dx[at], some)
    sums = torch.zeros(4, N, dtype=torch.float64, device=DEV)
    for i in range(0, R, 50000):
        d = dy[i:i + 50000].double()
        u = (x[i:i + 50000].double() - mean[i:i + 50000].double()[:, None]) * rstd[i:i + 50000].double()[:, None]
        sums += torch.stack([(d * u).sum(0), (d * u).abs().sum(0), d.sum(0), d.abs().sum(0)])
    sums = sums.cpu()
    chain = R / 256 + 200                             # rows of one group, its block's groups, the blocks' parts
    close(dw, sums[0], (chain + 4) * U * sums[1], torch.float32, "dweight")
    close(db, sums[2], chain * U * sums[3], torch.float32, "dbias")


def test_layer_norm_of_more_dimensions_and_views():
    g = rng(77)
    x = normal(g, 4, 6, 50).to(DEV)
    w = normal(g, 50).to(DEV)
    flat = G.layer_norm(x.view(24, 50), w)
    assert torch.equal(G.layer_norm(x, w), flat.view(4, 6, 50))
    assert torch.equal(G.layer_norm(x[0, 0], w), flat[0])
    assert torch.equal(G.layer_norm(x.transpose(0, 1), w), flat.view(4, 6, 50).transpose(0, 1))
    leaf = x.clone().requires_grad_()
    G.layer_norm(leaf.transpose(0, 1), w).sum().backward()      # the gradient is one broadcast value
    assert leaf.grad.shape == x.shape and bool(torch.isfinite(leaf.grad).all())


def test_layer_norm_passes_nan_and_inf_on_within_their_rows():
    x = torch.randn(5, 64, device=DEV)
    x[1, 3], x[3, 60] = float("nan"), float("inf")
    y = G.layer_norm(x)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all())
    assert bool(torch.isfinite(y[[0, 2, 4]]).all())


def test_gradients_that_are_not_asked_for_and_inputs_that_are_not_given():
    """Each subset of the inputs on its own gives the bits of all together."""
    g = rng(61)
    x, w, b, dy = (normal(g, *s).to(DEV).requires_grad_() for s in ((30, 70), (70,), (70,), (30, 70)))
    both = torch.autograd.grad(G.layer_norm(x, w, b), [x, w, b], dy)
    for i, leaf in enumerate((x, w, b)):
        assert torch.equal(torch.autograd.grad(G.layer_norm(x, w, b), leaf, dy)[0], both[i])
    alone, = torch.autograd.grad(G.layer_norm(x.detach(), None, b), b, dy)
    assert torch.equal(alone, both[2])
    dx, db = torch.autograd.grad(G.layer_norm(x, None, b), [x, b], dy)
    assert torch.equal(db, both[2]) and torch.equal(dx, torch.autograd.grad(G.layer_norm(x), x, dy)[0])
    assert torch.equal(torch.autograd.grad(G.layer_norm(x.detach(), w.detach(), b), b, dy)[0], both[2])

    r = G.RowRoute(torch.randint(0, 3, (30, 2), generator=g).to(DEV), 3)
    rows, wt = normal(g, 60, 70).to(DEV).requires_grad_(), torch.rand(30, 2, generator=g).to(DEV).requires_grad_()
    drows, dwt = torch.autograd.grad(G.combine(r, rows, wt), [rows, wt], dy)
    assert torch.equal(torch.autograd.grad(G.combine(r, rows, wt.detach()), rows, dy)[0], drows)
    assert torch.equal(torch.autograd.grad(G.combine(r, rows.detach(), wt), wt, dy)[0], dwt)
    assert torch.equal(torch.autograd.grad(G.combine(r, rows, wt), wt, dy)[0], dwt)
    m, o = normal(g, 3, 70, 20).to(DEV).requires_grad_(), torch.tensor([0, 5, 5, 28], device=DEV)
    d = dy[:, :20].detach()                           # a strided gradient
    dx, dm = torch.autograd.grad(G.segment_matmul(x, m, o), [x, m], d)
    assert torch.equal(torch.autograd.grad(G.segment_matmul(x, m.detach(), o), x, d)[0], dx)
    assert torch.equal(torch.autograd.grad(G.segment_matmul(x.detach(), m, o), m, d)[0], dm)


def test_broadcast_inputs_and_second_derivatives():
    g = rng(62)
    r = G.RowRoute(torch.randint(0, 3, (30, 2), generator=g).to(DEV), 3)
    rows, one = normal(g, 60, 8).to(DEV), torch.rand(30, 1, generator=g).to(DEV).requires_grad_()
    full = one.detach().expand(30, 2).contiguous().requires_grad_()
    out, want = G.combine(r, rows, one.expand(30, 2)), G.combine(r, rows, full)
    assert torch.equal(out, want)
    d1, = torch.autograd.grad(out.sum(), one)
    d2, = torch.autograd.grad(want.sum(), full)
    assert torch.equal(d1, d2.sum(1, keepdim=True))
    x = normal(g, 4, 8).to(DEV).requires_grad_()
    dx, = torch.autograd.grad(G.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        dx.sum().backward()
    with torch.no_grad():
        assert not G.layer_norm(x).requires_grad


# ------------------------------------------------------------------ together

def block(mod, p, expert, E):
    """Layer norm, the experts' two products with an activation between them,
    and the sum back."""
    x, gamma, beta, w1, w2, weight = p
    h = mod.layer_norm(x, gamma, beta, 1e-5)
    r = mod.RowRoute(expert, E)
    a = mod.segment_matmul(mod.dispatch(r, h), w1, r.offsets)
    z = mod.segment_matmul(a * torch.sigmoid(a), w2, r.offsets)
    return x + mod.combine(r, z, weight)


class Plain:
    """The same calls in 64 bits on the CPU, with torch's own gradients."""
    class RowRoute:
        def __init__(self, expert, E):
            self.expert, self.E = expert, E
            o, order, pos = plain_route(expert, E)
            self.offsets, self.order, self.position = (torch.from_numpy(np.ascontiguousarray(v)) for v in (o, order, pos))

    @staticmethod
    def layer_norm(x, w, b, eps):
        d = x - x.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + eps) * w + b

    @staticmethod
    def dispatch(r, x):
        live = torch.arange(r.order.numel()) < r.offsets[-1]
        return torch.where(live[:, None], x[r.order // r.expert.shape[1]], torch.zeros((), dtype=x.dtype))

    @staticmethod
    def segment_matmul(x, w, offsets):
        o = offsets.tolist()
        return torch.cat([x[o[e]:o[e + 1]] @ w[e] for e in range(len(o) - 1)] + [x[o[-1]:] @ w[0] * 0])

    @staticmethod
    def combine(r, rows, w):
        there = (r.position < r.offsets[-1])[:, :, None]
        return (w[:, :, None] * torch.where(there, rows[r.position], torch.zeros((), dtype=rows.dtype))).sum(1)


def block_inputs(seed=3, T=150, k=2, E=6, N=48, H=80):
    g = rng(seed, T)
    expert = pairs_of(g, T, k, E, "some")
    p = [normal(g, T, N), normal(g, N, scale=0.1, shift=1.0), normal(g, N, scale=0.1),
         normal(g, E, N, H, scale=N ** -0.5), normal(g, E, H, N, scale=H ** -0.5),
         torch.softmax(normal(g, T, k), 1)]
    return expert, p, normal(g, T, N), E


def test_block_of_all_operators_and_its_gradients():
    """Forward and every gradient against 64 bits.  Each of the ~8 operators
    on the way adds at most its sum length (at most 512 rows here) times u of
    the magnitudes it adds; taken together within 2^-24 * 8 * 512 = 2.5e-4 of
    each output's largest value."""
    expert, p, dout, E = block_inputs()
    leaves = [t.to(DEV).requires_grad_() for t in p]
    out = block(G, leaves, expert.to(DEV), E)
    grads = torch.autograd.grad(out, leaves, dout.to(DEV))
    ref = [t.double().requires_grad_() for t in p]
    want = block(Plain, ref, expert, E)
    wgrads = torch.autograd.grad(want, ref, dout.double())
    for got, w in zip([out, *grads], [want, *wgrads]):
        w = w.detach()
        assert float((got.detach().double().cpu() - w).abs().max()) <= 8 * 512 * U * float(w.abs().max())


def test_gradients_against_differences():
    """<gradient, v> against (f(p + h v) - f(p - h v)) / 2 h of the kernels'
    own forward, f = sum(c * out).  What the difference leaves out is computed
    in 64 bits (difference minus derivative of the plain form); what is left
    is rounding: f within 8 * 512 * u of sum|c * out| on each side."""
    expert, p, c, E = block_inputs(seed=8)
    h = 2.0 ** -7
    leaves = [t.to(DEV).requires_grad_() for t in p]
    ed, cd = expert.to(DEV), c.to(DEV).double()
    grads = torch.autograd.grad(block(G, leaves, ed, E), leaves, c.to(DEV))
    ref = [t.double().requires_grad_() for t in p]
    wgrads = torch.autograd.grad(block(Plain, ref, expert, E), ref, c.double())
    g = rng(55)
    for i in range(len(p)):
        # v and h * v are short binary fractions and the moved point is rounded
        # once, so the step taken is read back from the moved points
        v = normal(g, *p[i].shape)
        ends = [p[i] + h * v, p[i] - h * v]
        v = (ends[0].double() - ends[1].double()) / (2 * h)
        with torch.no_grad():
            f, f64, size = [], [], 0.0
            for q in ends:
                moved = [q.to(DEV) if j == i else t.detach() for j, t in enumerate(leaves)]
                out = block(G, moved, ed, E).double()
                f.append(float((cd * out).sum()))
                size += float((cd * out).abs().sum())
                m64 = [q.double() if j == i else t.detach() for j, t in enumerate(ref)]
                f64.append(float((c.double() * block(Plain, m64, expert, E)).sum()))
        left_out = abs((f64[0] - f64[1]) / (2 * h) - float((wgrads[i] * v).sum()))
        slope = float((grads[i].double().cpu() * v).sum())
        tol = left_out + 8 * 512 * U * size / (2 * h)
        assert abs(slope - (f[0] - f[1]) / (2 * h)) <= tol, (i, slope, (f[0] - f[1]) / (2 * h), tol)


def test_two_runs_give_the_same_bits():
    expert, p, dout, E = block_inputs(T=3000)
    leaves = [t.to(DEV).requires_grad_() for t in p]
    runs = []
    for _ in range(2):
        out = block(G, leaves, expert.to(DEV), E)
        runs.append([out.detach()] + list(torch.autograd.grad(out, leaves, dout.to(DEV))))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_block_captured_and_replayed_with_new_inputs():
    """Forward and backward in one graph, two of them alive at once; every
    replay follows the inputs that stand in its buffers."""
    expert, p, dout, E = block_inputs(T=200)
    graphs = []
    for n in range(2):
        static = [t.to(DEV).requires_grad_() for t in p]
        e, d = expert.to(DEV), dout.to(DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.autograd.grad(block(G, static, e, E), static, d)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            out = block(G, static, e, E)
            grads = torch.autograd.grad(out, static, d)
        graphs.append((graph, static, e, d, out, grads))
    for rep in range(4):
        for n, (graph, static, e, d, out, grads) in enumerate(graphs):
            ex, q, do, _ = block_inputs(seed=20 + 2 * rep + n, T=200)
            with torch.no_grad():
                for s, t in zip(static, q):
                    s.copy_(t)
                e.copy_(ex)
                d.copy_(do)
            _ = float(torch.randn(1 << 18, device=DEV).sum())
            graph.replay()
            torch.cuda.synchronize()
            leaves = [t.to(DEV).requires_grad_() for t in q]
            want = block(G, leaves, ex.to(DEV), E)
            wgrads = torch.autograd.grad(want, leaves, do.to(DEV))
            assert torch.equal(out, want), f"replay {rep} of graph {n}"
            assert all(torch.equal(a, b) for a, b in zip(grads, wgrads)), f"replay {rep} of graph {n}"


def test_captured_backward_beside_an_eager_graph_of_its_leaves_is_refused():
    """The gradient of a leaf whose eager graph lives would leave the capture;
    once that graph is gone, the same backward pass is captured and replayed."""
    g = rng(73)
    x, w = normal(g, 40, 24).to(DEV).requires_grad_(), normal(g, 3, 24, 16).to(DEV).requires_grad_()
    e = torch.randint(0, 3, (20, 2), generator=g).to(DEV)
    d40, d16 = normal(g, 40, 24).to(DEV), normal(g, 40, 16).to(DEV)
    weight = normal(g, 20, 2).to(DEV).requires_grad_()
    route = G.RowRoute(e, 3)
    x20 = normal(g, 20, 24).to(DEV).requires_grad_()
    d20, d80 = normal(g, 20, 24).to(DEV), normal(g, 40, 24).to(DEV)
    cases = [(lambda: G.layer_norm(x), x, d40), (lambda: G.segment_matmul(x.detach(), w, route.offsets), w, d16),
             (lambda: G.combine(route, x.detach(), weight), weight, d20), (lambda: G.dispatch(route, x20), x20, d80)]
    for call, leaf, d in cases:
        alive = call()
        want, = torch.autograd.grad(call(), leaf, d)
        torch.cuda.synchronize()
        refused = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="stream outside the capture"):
            with torch.cuda.graph(refused, capture_error_mode="thread_local"):
                torch.autograd.grad(call(), leaf, d)
        del alive
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            got, = torch.autograd.grad(call(), leaf, d)
        for _ in range(3):
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_another_stream():
    expert, p, dout, E = block_inputs(T=400)
    leaves = [t.to(DEV).requires_grad_() for t in p]
    want = block(G, leaves, expert.to(DEV), E)
    wgrads = torch.autograd.grad(want, leaves, dout.to(DEV))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = block(G, leaves, expert.to(DEV), E)
        grads = torch.autograd.grad(out, leaves, dout.to(DEV))
    side.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(grads, wgrads))


def test_aggregation_and_typed_product_together():
    """Neighbour aggregation, layer norm and a product per node type, as a
    relational graph layer runs them."""
    import workloads as W
    w = W.make("tiny")
    g = w.graph
    adj = G.SparseAdj(torch.from_numpy(g.rowptr).to(DEV), torch.from_numpy(g.col).to(DEV),
                      torch.from_numpy(g.val).to(DEV), num_cols=g.K)
    gen = rng(91)
    types = torch.randint(0, 4, (g.M,), generator=gen)
    wt = normal(gen, 4, w.B.shape[1], 24).to(DEV).requires_grad_()
    B = torch.from_numpy(w.B).to(DEV).requires_grad_()
    r = G.RowRoute(types.to(DEV), 4)
    h = G.layer_norm(G.aggregate(adj, B, "mean"))
    out = G.combine(r, G.segment_matmul(G.dispatch(r, h), wt, r.offsets))
    want = torch.einsum("mi,mio->mo", h.detach().double().cpu(), wt.detach().double().cpu()[types])
    assert float((out.detach().double().cpu() - want).abs().max()) <= 2 * U * 64 * 16 * float(want.abs().max())
    dB, dw = torch.autograd.grad(out.square().sum(), [B, wt])
    assert dB.shape == B.shape and bool(torch.isfinite(dB).all()) and bool(dB.any()) and bool(dw.any())
    adj.close()


def test_forward_mode_is_refused():
    """A tangent is refused whether or not gradients are recorded, never dropped."""
    g = rng(71)
    x, t = normal(g, 6, 8).to(DEV), normal(g, 6, 8).to(DEV)
    w, weight = normal(g, 2, 8, 4).to(DEV), normal(g, 6, 1).to(DEV)
    route = G.RowRoute(torch.tensor([0, 1, 1, 0, 1, 0], device=DEV).reshape(6, 1), 2)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, t)
        for call in (lambda: G.layer_norm(dual), lambda: G.dispatch(route, dual),
                     lambda: G.combine(route, dual, weight),
                     lambda: G.segment_matmul(dual, w, route.offsets)):
            with pytest.raises(RuntimeError, match="jvp"):
                call()
            with torch.no_grad(), pytest.raises(RuntimeError, match="jvp"):
                call()
    torch.testing.assert_close(G.layer_norm(x), torch.nn.functional.layer_norm(x, (8,)))
