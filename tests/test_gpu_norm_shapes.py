"""The layer norm at every shape of lanes and packs that its kernels have:
widths at, below and above each border, fewer rows than one block takes and
several rows for each group of lanes.

A row's sum is a chain of at most 64 + N / 1024 additions, the columns' sums
one of at most R / 256 + 200; u = 2^-24, first order, with the factor 1.01 for
the rest.  The formulas for the mean, the variance and what follows from them
count a rounding for every operation."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gnn_sparse_dense_amd as G
    from tests.gpu_helpers import DEV, log

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
PACK = {"fp32": 4, "bf16": 8, "fp16": 8}
U = 2.0 ** -24
EPS = 1e-5

# packs of 16 bytes at which a row goes to more lanes, or to the kernels for long rows
BORDERS = [4, 8, 16, 32, 64, 128, 256, 512, 1024, 2048, 4096]


def close(got, ref, before, dtype, what):
    err = (got.double() - ref).abs()
    f = torch.finfo(dtype)
    size = ref.abs() + before
    bad = ~(err <= 1.01 * (before + size * (f.eps / 2) + f.smallest_normal * f.eps / 2))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error {float(err.max()):.3e}"


def check(R, N, kind, wtype):
    dtype = TYPES[kind]
    g = torch.Generator(device=DEV)
    g.manual_seed(R + 31 * N)

    def normal(*shape, dtype=dtype, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype)
    x, dy = normal(R, N, scale=2.0, shift=0.5), normal(R, N)
    w, b = normal(N, dtype=wtype), normal(N, dtype=wtype)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = G.layer_norm(*leaves, eps=EPS)
    grads = torch.autograd.grad(y, leaves, dy)

    X, D, W, B = (t.detach().double() for t in (x, dy, w, b))
    mean = X.mean(1, keepdim=True)
    d = X - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    unit = d * rstd
    chain = 64 + N / 1024
    e_mean = (chain + 2) * U * X.abs().mean(1, keepdim=True)
    e_d = e_mean + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d * e_d).mean(1, keepdim=True) + (chain + 3) * U * var
    a = (e_var / (var + EPS)).clamp(max=0.5)
    e_rstd = (e_var / (2 * (var + EPS)) + 6 * U) * (1 - a) ** -1.5      # relative
    e_unit = e_d * rstd * (1 + e_rstd) + unit.abs() * (e_rstd + 2 * U)
    ref = unit * W + B
    close(y.detach(), ref, W.abs() * e_unit + 2 * U * ((W * unit).abs() + ref.abs()), dtype, "y")
    gr = D * W
    mg, mgu = gr.mean(1, keepdim=True), (gr * unit).mean(1, keepdim=True)
    e_mg = (chain + 3) * U * gr.abs().mean(1, keepdim=True)
    e_mgu = (gr.abs() * e_unit).mean(1, keepdim=True) + (chain + 4) * U * (gr * unit).abs().mean(1, keepdim=True)
    inner = gr - mg - unit * mgu
    e_dx = rstd * (1 + e_rstd) * (e_mg + unit.abs() * e_mgu + e_unit * (mgu.abs() + e_mgu)
                                  + 5 * U * (gr.abs() + mg.abs() + (unit * mgu).abs())) \
        + rstd * inner.abs() * (e_rstd + U)
    close(grads[0], rstd * inner, e_dx, dtype, "dx")
    rows = R / 256 + 200
    close(grads[1], (D * unit).sum(0), (D.abs() * e_unit).sum(0) + (rows + 4) * U * (D * unit).abs().sum(0), wtype, "dweight")
    close(grads[2], D.sum(0), rows * U * D.abs().sum(0), wtype, "dbias")


@pytest.mark.parametrize("kind,weights", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"),
                                          ("fp16", "fp16")])
@pytest.mark.parametrize("packs", BORDERS)
def test_layer_norm_around_each_border(packs, kind, weights):
    """Whole packs, one element more and one less; 37 rows end inside a block."""
    for more in (-1, 0, 1):
        log(f"norm N={packs * PACK[kind] + more} {kind} weights={weights}")
        check(37, packs * PACK[kind] + more, kind, TYPES[weights])


def rows_for_turns(packs):
    """More rows than two turns of every group take: the forward pass runs at
    most 32 waves (16 where a group is less than a wave) on each of 256 units,
    the backward pass fewer."""
    lanes = min(1024, max(4, packs if packs <= 64 else packs // 2))
    most = 256 * (16 if lanes < 64 else 32) * 64 // max(256, lanes) * max(1, 256 // lanes)
    return 2 * most + 3


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("packs", BORDERS)
def test_layer_norm_of_several_rows_to_a_group(packs, kind):
    """More than two rows to a group, up to 32 million elements (long rows: as many rows as that gives)."""
    N = packs * PACK[kind] - 3
    R = min(rows_for_turns(packs), (1 << 25) // N | 1)
    log(f"norm R={R} N={N} {kind}")
    check(R, N, kind, torch.float32)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("shift", [1, 3])
@pytest.mark.parametrize("N", [5, 72, 1024, 1027, 20001])
def test_layer_norm_at_any_alignment(N, shift, kind):
    """Rows and weights that start in the middle of a 16-byte group: the same bits as aligned ones."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N + shift)
    dtype = TYPES[kind]

    def moved(t):
        whole = torch.zeros(t.numel() + shift, dtype=t.dtype, device=DEV)
        whole[shift:] = t.reshape(-1)
        return whole[shift:].view(t.shape)
    x, dy, w, b = (torch.randn(*s, generator=g, device=DEV).to(dtype) for s in ((11, N), (11, N), (N,), (N,)))
    outs = []
    for m in (moved, lambda t: t.clone()):
        leaves = [m(t).requires_grad_() for t in (x, w, b)]
        y = G.layer_norm(*leaves)
        outs.append([y.detach(), *torch.autograd.grad(y, leaves, m(dy))])
    assert all(torch.equal(p, q) for p, q in zip(*outs))
