"""Backward passes of the layer norm that are captured into a graph: inputs of
any number of dimensions, and torch's own mode of capture."""
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
