"""Gradients of the row operators that are differentiated again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV
    from tests.test_gpu_rows import normal, rng


# -------------------------------------------------------- second derivatives

def again(outputs, inputs):
    """First derivatives of a sum, whose incoming gradient is a constant."""
    return torch.autograd.grad(outputs.sum(), inputs, create_graph=True)


def recorded(outputs, inputs):
    """First derivatives of a sum of squares, whose incoming gradient is recorded."""
    return torch.autograd.grad(outputs.square().sum(), inputs, create_graph=True)


def raises(grad, *others):
    """A penalty on grad, added to a loss that is differentiable without it."""
    assert grad.requires_grad
    loss = grad.square().sum() + sum(o.square().sum() for o in others)
    for ask in (lambda: torch.autograd.grad(loss, others, retain_graph=True), lambda: loss.backward(inputs=others)):
        with pytest.raises(RuntimeError, match="differentiable once"):
            ask()


def test_second_derivatives_through_saved_inputs_raise():
    """dx of a product depends on w, and so on: with a constant incoming
    gradient too, differentiating it raises and is not taken as zero."""
    g = rng(81)
    x, w = normal(g, 20, 8).to(DEV).requires_grad_(), normal(g, 2, 8, 4).to(DEV).requires_grad_()
    o = torch.tensor([0, 9, 18], device=DEV)
    for wanted in ([x], [w], [x, w]):
        for grad in again(G.segment_matmul(x, w, o), wanted):
            raises(grad, x, w)
    r = G.RowRoute(torch.randint(0, 3, (10, 2), generator=g).to(DEV), 3)
    rows, weight = normal(g, 20, 8).to(DEV).requires_grad_(), torch.rand(10, 2, generator=g).to(DEV).requires_grad_()
    for wanted in ([rows], [weight], [rows, weight]):
        for grad in again(G.combine(r, rows, weight), wanted):
            raises(grad, rows, weight)
    gamma, beta = normal(g, 8).to(DEV).requires_grad_(), normal(g, 8).to(DEV).requires_grad_()
    for grad in again(G.layer_norm(x, gamma, beta), [x, gamma]):
        raises(grad, x, gamma)
    raises(again(G.layer_norm(x), x)[0], x)
    raises(again(G.layer_norm(x, None, beta), x)[0], x)
    raises(again(G.layer_norm(x.reshape(4, 5, 8), gamma), x)[0], x)


def test_second_derivatives_through_recorded_gradients_raise():
    """Also where only an input's gradient is asked for: the way to what raises
    is then a part of the graph that reaches the input."""
    g = rng(83)
    x, w = normal(g, 20, 8).to(DEV).requires_grad_(), normal(g, 2, 8, 4).to(DEV).requires_grad_()
    o = torch.tensor([0, 9, 18], device=DEV)
    r = G.RowRoute(torch.randint(0, 3, (20, 2), generator=g).to(DEV), 3)
    rows, weight = normal(g, 40, 8).to(DEV).requires_grad_(), torch.rand(20, 2, generator=g).to(DEV).requires_grad_()
    beta = normal(g, 8).to(DEV).requires_grad_()
    raises(recorded(G.dispatch(r, x), x)[0], x)
    raises(recorded(G.combine(r, rows), rows)[0], rows)
    raises(recorded(G.layer_norm(x), x)[0], x)
    for grad in recorded(G.combine(r, rows, weight), [rows, weight]):
        raises(grad, rows, weight)
    for grad in recorded(G.segment_matmul(x, w, o), [x, w]):
        raises(grad, x, w)
    for grad in recorded(G.layer_norm(x, None, beta), [x, beta]):
        raises(grad, x, beta)


def test_gradients_that_are_constants_stay_so():
    """What no recorded input moves can stand beside a graph: the gradients of
    dispatch, of the layer norm's bias and of inputs whose partner needs none."""
    g = rng(82)
    x, w = normal(g, 20, 8).to(DEV).requires_grad_(), normal(g, 2, 8, 4).to(DEV).requires_grad_()
    o = torch.tensor([0, 9, 18], device=DEV)
    r = G.RowRoute(torch.randint(0, 3, (10, 2), generator=g).to(DEV), 3)
    x10, rows = normal(g, 10, 8).to(DEV).requires_grad_(), normal(g, 20, 8).to(DEV).requires_grad_()
    weight = torch.rand(10, 2, generator=g).to(DEV).requires_grad_()
    gamma, beta = normal(g, 8).to(DEV).requires_grad_(), normal(g, 8).to(DEV).requires_grad_()
    cases = [(lambda: G.dispatch(r, x10), x10), (lambda: G.combine(r, rows), rows),
             (lambda: G.combine(r, rows, weight.detach()), rows), (lambda: G.combine(r, rows.detach(), weight), weight),
             (lambda: G.segment_matmul(x, w.detach(), o), x), (lambda: G.segment_matmul(x.detach(), w, o), w),
             (lambda: G.layer_norm(x, gamma, beta), beta), (lambda: G.layer_norm(x.detach(), gamma, beta), gamma)]
    for call, leaf in cases:
        want, = torch.autograd.grad(call().sum(), leaf)
        got, = again(call(), leaf)
        assert not got.requires_grad and torch.equal(got, want)
    # recorded or not, the first derivatives are the same bits
    leaves = [x, gamma, beta]
    for a, b in zip(again(G.layer_norm(*leaves), leaves), torch.autograd.grad(G.layer_norm(*leaves).sum(), leaves)):
        assert torch.equal(a.detach(), b)
