"""Attention within segments, dropout and the loss as a training step runs them,
next to the layer norm, the experts' products and the aggregation: together, on
streams, captured, and what is refused."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests import rows64  # noqa: E402
from tests.test_gpu_rows import normal, pairs_of, rng  # noqa: E402

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV

P, SEED = 0.2, 41
H, D, E, V = 4, 8, 3, 21


def inputs(seed=1, lengths=(40, 1, 59)):
    """Parameters, offsets, experts and targets of one block over packed rows of 32."""
    g, N = rng(seed, *lengths), H * D
    T = sum(lengths) + 3
    offsets = torch.tensor([0] + list(np.cumsum(lengths)))
    expert = pairs_of(g, T, 2, E, "some")
    target = torch.where(torch.rand(T, generator=g) < 0.3, torch.tensor(-1), torch.randint(0, V, (T,), generator=g))
    p = [normal(g, T, N), normal(g, N, scale=0.1, shift=1.0), normal(g, N, scale=0.1), normal(g, 1, N, 2 * N, scale=N ** -0.5),
         normal(g, E, N, N, scale=N ** -0.5), torch.softmax(normal(g, T, 2), 1), normal(g, V, N, scale=N ** -0.5)]
    return p, offsets, expert, target


def step(p, offsets, expert, target, seed):
    """Norm, attention (two key heads for four), dropout into the residual, the
    experts, dropout again, loss."""
    x, gamma, beta, wqkv, we, weight, w = p
    T, N = x.shape
    h = G.layer_norm(x, gamma, beta)
    whole = torch.tensor([0, T], device=x.device) if not isinstance(offsets, tuple) else offsets[1]
    bounds = offsets[0] if isinstance(offsets, tuple) else offsets
    qkv = G.segment_matmul(h, wqkv, whole)
    q, k, v = qkv.split([N, N // 2, N // 2], 1)
    a = G.segment_attention(q.unflatten(1, (H, D)), k.unflatten(1, (H // 2, D)), v.unflatten(1, (H // 2, D)), bounds,
                            causal=True)
    x = G.dropout(a.flatten(1), P, seed, 0, x)
    r = G.RowRoute(expert, E)
    z = G.segment_matmul(G.dispatch(r, x), we, r.offsets)
    x = G.dropout(G.combine(r, z, weight), P, seed, 1, x)
    return G.linear_cross_entropy(x, w, target)


def plain_step(p, offsets, expert, target, seed):
    """The same in 64 bits on the CPU, with torch's own gradients."""
    x, gamma, beta, wqkv, we, weight, w = p
    T, N = x.shape
    c = x - x.mean(1, keepdim=True)
    h = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * gamma + beta
    q, k, v = (h @ wqkv[0]).split([N, N // 2, N // 2], 1)
    o, outs = offsets.tolist(), []
    for a, b in zip(o, o[1:]):
        late = torch.ones(b - a, b - a, dtype=torch.bool).triu(1)
        heads = []
        for i in range(H):
            qs, ks, vs = q[a:b, i * D:(i + 1) * D], k[a:b, i // 2 * D:(i // 2 + 1) * D], v[a:b, i // 2 * D:(i // 2 + 1) * D]
            heads.append(torch.softmax((qs @ ks.T * D ** -0.5).masked_fill(late, -1e30), 1) @ vs)
        outs.append(torch.cat(heads, 1))
    outs.append(torch.zeros(T - o[-1], N, dtype=torch.float64))
    keep = [rows64.kept(T * N, P, seed, i).view(T, N).double() / (1 - P) for i in (0, 1)]
    x = x + keep[0] * torch.cat(outs)
    z = torch.zeros_like(x)
    for j in range(2):
        e = expert[:, j]
        live = ((e >= 0) & (e < E)).double()
        z = z + (weight[:, j] * live)[:, None] * torch.einsum("ti,tio->to", x, we[e.clamp(0, E - 1)])
    x = x + keep[1] * z
    return torch.nn.functional.cross_entropy(x @ w.T, torch.where(target < 0, torch.tensor(-100), target))


def test_step_and_its_gradients():
    """Forward and every gradient against 64 bits.  Each of the ~12 operators on the
    way adds at most its sum length (at most 103 rows here, 64 elements) times 2 u of
    the magnitudes it adds, in both passes; taken together within 24 * 2 * 103 * u =
    2.9e-4 of each output's largest value."""
    p, offsets, expert, target = inputs()
    leaves = [t.to(DEV).requires_grad_() for t in p]
    loss = step(leaves, offsets.to(DEV), expert.to(DEV), target.to(DEV), torch.tensor([SEED], device=DEV))
    grads = torch.autograd.grad(loss, leaves)
    ref = [t.double().requires_grad_() for t in p]
    want = plain_step(ref, offsets, expert, target, SEED)
    for got, w in zip([loss, *grads], [want, *torch.autograd.grad(want, ref)]):
        w = w.detach()
        assert float((got.detach().double().cpu() - w).abs().max()) <= 24 * 2 * 103 * rows64.U * float(w.abs().max())


def test_step_behind_the_aggregation():
    import workloads as W
    w = W.make("tiny")
    g = w.graph
    adj = G.SparseAdj(torch.from_numpy(g.rowptr).to(DEV), torch.from_numpy(g.col).to(DEV),
                      torch.from_numpy(g.val).to(DEV), num_cols=g.K)
    B = torch.from_numpy(w.B).to(DEV).requires_grad_()
    h = G.dropout(G.aggregate(adj, B, "mean"), 0.5, 3)
    M, N = h.shape
    a = G.segment_attention(h.view(M, 1, N), h.view(M, 1, N), h.view(M, 1, N), torch.tensor([0, M // 2, M], device=DEV))
    classes = normal(rng(5), 7, N).to(DEV)
    loss = G.linear_cross_entropy(a.view(M, N), classes, torch.arange(M, device=DEV) % 7)
    dB, = torch.autograd.grad(loss, B)
    assert bool(torch.isfinite(loss.detach())) and bool(torch.isfinite(dB).all()) and bool(dB.any())
    adj.close()


def gpu(p, offsets, expert, target):
    return ([t.to(DEV).requires_grad_() for t in p], offsets.to(DEV), expert.to(DEV), target.to(DEV))


def run(args, seed):
    loss = step(*args, seed)
    return [loss, *torch.autograd.grad(loss, args[0])]


def test_same_bits_again_and_on_another_stream():
    args, seed = gpu(*inputs(2, (300, 5, 400))), torch.tensor([SEED], device=DEV)
    want = run(args, seed)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run(args, seed), want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run(args, seed)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    both = []                                          # two calls at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.no_grad():
            both.append(step(*args, seed))
    torch.cuda.synchronize()
    assert all(torch.equal(b, want[0]) for b in both)


def test_captured_and_replayed_with_new_inputs():
    """Forward and backward in one graph, two of them alive at once; every replay
    follows the inputs, offsets, targets and seed that stand in its buffers."""
    graphs = []
    for n in range(2):
        p, offsets, expert, target = inputs(3)
        static, o, e, t = gpu(p, offsets, expert, target)
        whole, seed = torch.tensor([0, p[0].shape[0]], device=DEV), torch.tensor([SEED], device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run((static, (o, whole), e, t), seed)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            got = run((static, (o, whole), e, t), seed)
        graphs.append((graph, static, o, e, t, seed, got, whole))
    for rep in range(3):
        for n, (graph, static, o, e, t, seed, got, _) in enumerate(graphs):
            lengths = [(40, 1, 59), (0, 100, 0), (33, 33, 34)][(rep + n) % 3]
            p, offsets, expert, target = inputs(10 + 2 * rep + n, lengths)
            with torch.no_grad():
                for s, v in zip(static, p):
                    s.copy_(v)
                o.copy_(offsets), e.copy_(expert), t.copy_(target), seed.fill_(100 + rep)
            float(torch.randn(1 << 18, device=DEV).sum())
            graph.replay()
            torch.cuda.synchronize()
            want = run(gpu(p, offsets, expert, target), torch.tensor([100 + rep], device=DEV))
            assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {rep} of graph {n}"


def calls():
    """Each operator with its inputs that take a gradient."""
    g = rng(60)
    q, k, v = (normal(g, 50, h, 16).to(DEV).requires_grad_() for h in (4, 2, 2))
    x, r, w = (normal(g, n, 24).to(DEV).requires_grad_() for n in (30, 30, 9))
    o, t = torch.tensor([0, 20, 50], device=DEV), torch.randint(0, 9, (30,), generator=g).to(DEV)
    seed = torch.tensor([7], device=DEV)
    return [(lambda: G.segment_attention(q, k, v, o), [q, k, v]), (lambda: G.dropout(x, 0.5, seed, 1, r), [x, r]),
            (lambda: G.dropout(x, 0.5, seed), [x]), (lambda: G.linear_cross_entropy(x, w, t, "none"), [x, w])]


def test_second_derivatives_raise():
    for call, leaves in calls():
        y = call()
        grads = torch.autograd.grad(y, leaves, torch.ones_like(y), create_graph=True)
        for leaf, d in zip(leaves, grads):
            if d.requires_grad:
                with pytest.raises(RuntimeError, match="differentiable once"):
                    torch.autograd.grad(d.sum(), leaf, allow_unused=True)
    x = torch.ones(8, device=DEV, requires_grad=True)       # linear: the gradient of dy is another call
    dy = torch.ones(8, device=DEV, requires_grad=True)
    d, = torch.autograd.grad(G.dropout(x, 0.5, 3), x, dy, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(d.sum(), dy)


def test_forward_mode_is_refused():
    with torch.autograd.forward_ad.dual_level():
        q = torch.autograd.forward_ad.make_dual(torch.ones(4, 1, 8, device=DEV), torch.ones(4, 1, 8, device=DEV))
        x = torch.autograd.forward_ad.make_dual(torch.ones(4, 8, device=DEV), torch.ones(4, 8, device=DEV))
        plain, o = torch.ones(4, 1, 8, device=DEV), torch.tensor([0, 4], device=DEV)
        t, w = torch.zeros(4, dtype=torch.int64, device=DEV), torch.ones(3, 8, device=DEV)
        for call in (lambda: G.segment_attention(q, plain, plain, o), lambda: G.segment_attention(plain, plain, q, o),
                     lambda: G.dropout(x, 0.5, 1), lambda: G.dropout(w.new_ones(4, 8), 0.5, 1, residual=x),
                     lambda: G.linear_cross_entropy(x, w, t), lambda: G.linear_cross_entropy(w.new_ones(4, 8), x, t)):
            with pytest.raises(RuntimeError, match="jvp"):
                call()
            with torch.no_grad(), pytest.raises(RuntimeError, match="jvp"):
                call()


def test_captured_backward_beside_an_eager_graph_is_refused():
    """And is captured and replayed once that graph is gone."""
    for call, leaves in calls():
        dy = torch.ones_like(call())
        alive = call()
        want = torch.autograd.grad(call(), leaves, dy)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="stream outside the capture"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), capture_error_mode="thread_local"):
                torch.autograd.grad(call(), leaves, dy)
        del alive
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode="thread_local"):
            got = torch.autograd.grad(call(), leaves, dy)
        for _ in range(3):
            for t in got:
                t.zero_() if t is not dy else None
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not dy)


def test_gradients_that_are_not_asked_for():
    for call, leaves in calls():
        y = call()
        dy = torch.ones_like(y)
        whole = torch.autograd.grad(y, leaves, dy, retain_graph=True)
        for i, leaf in enumerate(leaves):
            assert torch.equal(torch.autograd.grad(y, leaf, dy, retain_graph=True)[0], whole[i])
        for i, leaf in enumerate(leaves):
            leaf.requires_grad_(False)
            if len(leaves) > 1:
                others = [t for t in leaves if t is not leaf]
                assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(call(), others, dy),
                                                             [w for j, w in enumerate(whole) if j != i]))
            leaf.requires_grad_(True)


def test_shapes_devices_and_values_are_refused():
    q, k, o = torch.ones(6, 4, 8, device=DEV), torch.ones(6, 2, 8, device=DEV), torch.tensor([0, 6], device=DEV)
    bad = [lambda: G.segment_attention(q, k[:, :, :4], k, o), lambda: G.segment_attention(q, k, k[:5], o),
           lambda: G.segment_attention(q[:5], k, k, o), lambda: G.segment_attention(q, k, k, o[:1]),
           lambda: G.segment_attention(q, k, k, o, torch.tensor([0, 3, 6], device=DEV)),
           lambda: G.segment_attention(q, k, k, o.cpu()), lambda: G.dropout(q, 0.5, torch.tensor([1])),
           lambda: G.dropout(q, 0.5, torch.tensor([1, 2], device=DEV)), lambda: G.dropout(q, 0.5, 1, residual=q[:5]),
           lambda: G.linear_cross_entropy(q[0], k[0], torch.zeros(3, dtype=torch.int64, device=DEV)),
           lambda: G.linear_cross_entropy(q[0], k[0], torch.zeros(4, dtype=torch.int64, device=DEV), "median"),
           lambda: G.linear_cross_entropy(q[0], torch.ones(3, 9, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: G.segment_attention(q, k, k, o.int()), lambda: G.dropout(q, 0.5, torch.tensor([1.0], device=DEV)),
                 lambda: G.dropout(q, 0.5, 1, residual=q.half()),
                 lambda: G.linear_cross_entropy(q[0], k[0], torch.zeros(4, device=DEV))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: G.segment_attention(q, q[:, :3], q[:, :3], o), lambda: G.segment_attention(q, k, k, o, scale=-1.0),
                 lambda: G.segment_attention(q, k, k, o, scale=0.0), lambda: G.dropout(q, 1.5, 1),
                 lambda: G.segment_attention(*(torch.ones(6, 1, 129, device=DEV),) * 3, o)):
        with pytest.raises(G.SpmmError):
            call()
