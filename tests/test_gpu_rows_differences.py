"""Gradients of the row operators together against differences of the kernels'
own forward, along directions in which the outputs' moves add up."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV
    from tests.test_gpu_rows import Plain, U, block, block_inputs, normal, rng


def forward_error(p, expert, E):
    """How far the block's outputs may be off, element by element: each
    operator's own roundings (u = 2^-24 each, two for a term of a matrix
    product) and what it hands on of its input's error, in 64 bits."""
    x, gamma, beta, w1, w2, weight = (t.double() for t in p)
    r = Plain.RowRoute(expert, E)
    n, hidden, k, chain = x.shape[1], w1.shape[2], weight.shape[1], 64
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-5)
    e_d = (chain + 2) * U * x.abs().mean(1, keepdim=True) + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d * e_d).mean(1, keepdim=True) + (chain + 3) * U * var
    e_rstd = (e_var / (2 * (var + 1e-5)) + 6 * U) * 1.01
    unit = d * rstd
    h = unit * gamma + beta
    e_h = gamma.abs() * (e_d * rstd * 1.01 + unit.abs() * (e_rstd + 2 * U)) + 2 * U * ((gamma * unit).abs() + h.abs())

    def product(rows, e_rows, w):
        e = Plain.segment_matmul(e_rows + 2 * U * w.shape[1] * (rows.abs() + e_rows), w.abs(), r.offsets)
        return Plain.segment_matmul(rows, w, r.offsets), e
    a, e_a = product(Plain.dispatch(r, h), Plain.dispatch(r, e_h), w1)
    s = a * torch.sigmoid(a)
    e_s = 1.1 * e_a + 12 * U * s.abs()               # |s'| < 1.1; exp, sum, quotient and product
    z, e_z = product(s, e_s, w2)
    out = x + Plain.combine(r, z, weight)
    return Plain.combine(r, e_z + k * U * (z.abs() + e_z), weight.abs()) + U * out.abs()


def test_gradients_against_differences_that_add_up():
    """<gradient, v> of f = sum(c * out) for random v, with c the signs of how
    each output moves along v, so that nothing cancels in the slope, against
    the difference of the kernels' own forward over 2 h.  What the difference
    takes beyond the slope is computed in 64 bits and taken off; what is left
    is rounding: of the outputs at both ends (element by element, above) and of
    the gradient (8 * 512 * u of its largest value for each element, as for the
    block).  That is below 1% of the slope, so a gradient 3% too large or too
    small is rejected, and so is one of zeros."""
    expert, p, _, E = block_inputs(seed=8)
    h, g = 0.25, rng(56)
    ed = expert.to(DEV)
    for i in range(len(p)):
        v = normal(g, *p[i].shape)
        ends = [p[i] + h * v, p[i] - h * v]
        v = (ends[0].double() - ends[1].double()) / (2 * h)          # the step that is taken
        with torch.no_grad():
            near = [block(Plain, [t.double() + (s * 2.0 ** -16 * v if j == i else 0) for j, t in enumerate(p)], expert, E)
                    for s in (1, -1)]
        c = torch.sign(near[0] - near[1])
        leaves = [t.to(DEV).requires_grad_() for t in p]
        grad, = torch.autograd.grad(block(G, leaves, ed, E), leaves[i], c.float().to(DEV))
        ref = [t.double().requires_grad_() for t in p]
        wgrad, = torch.autograd.grad(block(Plain, ref, expert, E), ref[i], c)
        f, f64, rounding = [], [], 0.0
        with torch.no_grad():
            for q in ends:
                moved = [(q if j == i else t).to(DEV) for j, t in enumerate(p)]
                f.append(float((c.to(DEV) * block(G, moved, ed, E).double()).sum()))
                moved = [(q if j == i else t).double() for j, t in enumerate(p)]
                f64.append(float((c * block(Plain, moved, expert, E)).sum()))
                rounding += 1.01 * float((c.abs() * forward_error(moved, expert, E)).sum())
        beyond = (f64[0] - f64[1]) / (2 * h) - float((wgrad * v).sum())
        want = (f[0] - f[1]) / (2 * h) - beyond
        slope = float((grad.double().cpu() * v).sum())
        tol = rounding / (2 * h) + 8 * 512 * U * float(wgrad.abs().max()) * float(v.abs().sum())
        assert tol < 0.01 * abs(want), (i, tol, want)
        assert abs(slope - want) <= tol, (i, slope, want, tol)
        assert min(abs(1.03 * slope - want), abs(0.97 * slope - want), abs(want)) > tol
