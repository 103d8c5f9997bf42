"""The plain forms in 64 bits that the row operators are compared with: pinned by
torch's own rules for gradients and by published values, on the CPU."""
import numpy as np
import torch

from tests import rows64


def test_generator_against_published_vectors():
    """Known answers of Philox 4x32 with 10 rounds (Salmon et al. 2011)."""
    zeros = rows64.philox(np.zeros((1, 4), dtype=np.uint64), 0, 0)[0]
    assert [f"{int(w):08x}" for w in zeros] == ["6627e8d5", "e169c58d", "bc57ac4c", "9b00dbd8"]
    ones = rows64.philox(np.full((1, 4), 0xFFFFFFFF, dtype=np.uint64), 0xFFFFFFFF, 0xFFFFFFFF)[0]
    assert [f"{int(w):08x}" for w in ones] == ["408f276d", "41c83b0e", "a20bc7c6", "6d5451fd"]


def test_attention_against_torch():
    g = torch.Generator().manual_seed(3)
    rows, keys = [2, 7, 7, 16], [0, 3, 9, 21]
    q = torch.randn(18, 4, 5, generator=g, dtype=torch.float64).requires_grad_()
    k = torch.randn(22, 2, 5, generator=g, dtype=torch.float64).requires_grad_()
    v = torch.randn(22, 2, 5, generator=g, dtype=torch.float64).requires_grad_()
    dout = torch.randn(18, 4, 5, generator=g, dtype=torch.float64)
    for causal in (False, True):
        outs = torch.zeros(18, 4, 5, dtype=torch.float64)
        for a, b, c, d in zip(rows, rows[1:], keys, keys[1:]):
            late = torch.zeros(b - a, d - c, dtype=torch.bool)
            if causal:
                late = torch.arange(d - c)[None, :] > torch.arange(b - a)[:, None] + (d - c) - (b - a)
            for h in range(4):
                s = (0.3 * q[a:b, h] @ k[c:d, h // 2].T).masked_fill(late, -1e30)
                p = torch.softmax(s, 1) * ~late
                outs = outs.index_put((torch.arange(a, b), torch.tensor(h)), p @ v[c:d, h // 2])
        want = [outs.detach(), *torch.autograd.grad(outs, [q, k, v], dout)]
        got = rows64.attention(q.detach().float(), k.detach().float(), v.detach().float(), rows, keys, causal, 0.3,
                               dout.float())
        for (value, bound), w in zip(got, want):
            assert float((value - w).abs().max()) < 1e-5 and bool((bound >= 0).all())


def test_loss_against_torch():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 6, generator=g).requires_grad_()
    w = torch.randn(5, 6, generator=g).requires_grad_()
    target = torch.tensor([0, 4, -1, 2, 5, 1, 1, -100, 3])
    ignored = torch.where((target < 0) | (target >= 5), torch.full_like(target, -100), target)
    for reduction in ("none", "sum", "mean"):
        want = torch.nn.functional.cross_entropy((x.double() @ w.double().T), ignored, reduction=reduction, ignore_index=-100)
        dloss = torch.rand(want.shape, generator=g)
        grads = torch.autograd.grad(want, [x, w], dloss.double())
        got = rows64.loss(x.detach(), w.detach(), target, reduction, dloss)
        for (value, bound), t in zip(got, [want.detach(), *grads]):
            assert float((value - t).abs().max()) < 1e-6 and bool((bound >= 0).all())
