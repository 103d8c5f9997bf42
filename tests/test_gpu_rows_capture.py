"""Backward passes of the row operators that are captured into a graph, in
torch's own mode of capture: inputs of any number of dimensions, and leaves
behind torch's operations."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV
    from tests.test_gpu_rows import normal, rng

SHAPES = [(24,), (40, 24), (4, 10, 24), (2, 3, 5, 24), (0, 3, 8)]


@pytest.mark.parametrize("shape", SHAPES)
def test_layer_norm_stands_next_to_its_leaves(shape):
    """No other node between the operator's and the leaf's, whose stream it looks at."""
    x, w = normal(rng(74), *shape).to(DEV).requires_grad_(), normal(rng(75), shape[-1]).to(DEV).requires_grad_()
    y = G.layer_norm(x, w)
    assert y.shape == x.shape
    assert [f.variable is t for (f, _), t in zip(y.grad_fn.next_functions, (x, w))] == [True, True]
    dy = normal(rng(76), *shape).to(DEV)
    dx, dw = torch.autograd.grad(y, [x, w], dy)
    flat = x.detach().reshape(-1, shape[-1]).requires_grad_()
    want = torch.autograd.grad(G.layer_norm(flat, w), [flat, w], dy.reshape(flat.shape))
    assert dx.shape == x.shape and torch.equal(dx.reshape(flat.shape), want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("shape", [s for s in SHAPES if len(s) != 2 and 0 not in s])
def test_captured_backward_beside_an_eager_graph_is_refused_in_any_dimensions(shape):
    x, dy = normal(rng(74), *shape).to(DEV).requires_grad_(), normal(rng(76), *shape).to(DEV)
    alive = G.layer_norm(x)
    want, = torch.autograd.grad(G.layer_norm(x), x, dy)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="stream outside the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(G.layer_norm(x), x, dy)
    del alive
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(G.layer_norm(x), x, dy)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_captured_backward_to_leaves_behind_torch_operations_is_refused():
    """The eager graph's leaf stands behind a cast, a product or a reshape."""
    g = rng(77)
    x, w = normal(g, 20, 24).to(DEV).requires_grad_(), normal(g, 3, 24, 16).to(DEV).requires_grad_()
    weight = normal(g, 20, 2).to(DEV).requires_grad_()
    r = G.RowRoute(torch.randint(0, 3, (20, 2), generator=g).to(DEV), 3)
    rows = normal(g, 40, 24).to(DEV)
    half, d24, d40 = torch.bfloat16, normal(g, 20, 24).to(DEV), normal(g, 40, 24).to(DEV)
    d16 = normal(g, 40, 16).to(DEV).to(half)
    cases = [(lambda: G.layer_norm(x * 2), x, d24), (lambda: G.layer_norm((x * 2).view(2, 10, 24)), x, d24.view(2, 10, 24)),
             (lambda: G.segment_matmul(rows.to(half), w.to(half), r.offsets), w, d16),
             (lambda: G.combine(r, rows, torch.softmax(weight, 1)), weight, d24), (lambda: G.dispatch(r, x + 1), x, d40)]
    for call, leaf, d in cases:
        alive = leaf * 1
        want, = torch.autograd.grad(call(), leaf, d)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="stream outside the capture"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                torch.autograd.grad(call(), leaf, d)
        del alive
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, = torch.autograd.grad(call(), leaf, d)
        for _ in range(3):
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_captured_backward_to_an_eager_result_is_refused():
    """The gradient of what was computed outside the capture goes to a node of
    that stream; the same values as a leaf of their own are captured."""
    x, d = normal(rng(78), 20, 24).to(DEV).requires_grad_(), normal(rng(79), 20, 24).to(DEV)
    eager = x * 2
    want, = torch.autograd.grad(G.layer_norm(eager), eager, d, retain_graph=True)
    torch.cuda.synchronize()
    for wanted in (eager, x):
        with pytest.raises(RuntimeError, match="stream outside the capture"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                torch.autograd.grad(G.layer_norm(eager), wanted, d, retain_graph=True)
        torch.cuda.synchronize()
    leaf = eager.detach().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, = torch.autograd.grad(G.layer_norm(leaf), leaf, d)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_a_layer_through_torchs_graphed_callables():
    """Forward and backward captured apart by torch, parameters as leaves."""
    class Layer(torch.nn.Module):
        def __init__(self, g):
            super().__init__()
            self.gamma, self.beta = (torch.nn.Parameter(normal(g, 24).to(DEV)) for _ in range(2))
            self.w = torch.nn.Parameter(normal(g, 3, 24, 16).to(DEV))

        def forward(self, x, expert, weight):
            r = G.RowRoute(expert, 3)
            h = G.layer_norm(x, self.gamma, self.beta)
            return G.combine(r, G.segment_matmul(G.dispatch(r, h), self.w, r.offsets), torch.softmax(weight, 1))

    def inputs(g):
        return (normal(g, 50, 24).to(DEV).requires_grad_(), torch.randint(-1, 3, (50, 2), generator=g).to(DEV),
                normal(g, 50, 2).to(DEV).requires_grad_())
    eager, layer = Layer(rng(91)), Layer(rng(91))
    graphed = torch.cuda.make_graphed_callables(layer, inputs(rng(92)))
    for seed in range(93, 97):
        got, want = inputs(rng(seed)), inputs(rng(seed))
        d = normal(rng(seed + 50), 50, 16).to(DEV)
        out, ref = graphed(*got), eager(*want)
        for m in (layer, eager):
            m.zero_grad()
        out.backward(d)
        ref.backward(d)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        pairs = [(got[0], want[0]), (got[2], want[2]), *zip(layer.parameters(), eager.parameters())]
        assert all(torch.equal(a.grad, b.grad) for a, b in pairs)


def test_captured_backward_beside_an_eager_graph_of_another_stream():
    """A leaf whose graph of a warm-up lives: its stream joins the capture."""
    x, d = normal(rng(95), 20, 24).to(DEV).requires_grad_(), normal(rng(96), 20, 24).to(DEV)
    w = normal(rng(97), 24).to(DEV).requires_grad_()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        alive = G.layer_norm(x, w)
        want = torch.autograd.grad(alive, [x, w], d, retain_graph=True)
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(G.layer_norm(x, w), [x, w], d)
    for _ in range(3):
        for t in got:
            t.zero_()
        float(torch.randn(1 << 16, device=DEV).sum())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del alive
