"""Attention within segments, dropout and the loss of a linear classifier, without a
GPU: sizes, types and arrays that are refused before the device is touched, and
the workspace calls."""
import ctypes

import pytest
import torch

import gnn_sparse_dense_amd as G

BIG = 2 ** 31
INV, UNS = G.SPMM_E_INVALID_ARG, G.SPMM_E_UNSUPPORTED
n = None


def refused(status, call, *args):
    assert getattr(G.lib(), call)(*args) == status, G.spmm_last_error()
    return G.spmm_last_error()[1]


def sizes(call, *args, outputs=1):
    out = [ctypes.c_int64(-1) for _ in range(outputs)]
    assert getattr(G.lib(), call)(*args, *(ctypes.byref(o) for o in out)) == G.SPMM_OK, G.spmm_last_error()
    return out[0].value if outputs == 1 else [o.value for o in out]


def attention(R=4, K=4, S=1, H=2, Hk=1, D=8, ldq=16, ldk=8, ldv=8, scale=1.0, kind=0, ws=n, bytes_=0):
    return (n, ldq, n, ldk, n, ldv, n, n, n, n, n, R, K, S, H, Hk, D, scale, 0, kind, ws, bytes_, n)


def backward(R=4, K=4, S=1, H=2, Hk=1, D=8, ldq=16, ldk=8, ldv=8, scale=1.0, kind=0, dq=64, ws=n, bytes_=0):
    return (n, ldq, n, ldk, n, ldv, n, n, n, n, n, n, dq, n, n, R, K, S, H, Hk, D, scale, 0, kind, ws, bytes_, n)


def test_attention_workspaces():
    call, back = "spmm_segment_attention_workspace", "spmm_segment_attention_backward_workspace"
    assert sizes(call, 8192, 8192, 3, 16, 4, 128, G.SPMM_BF16) == 0              # tiles enough
    few = sizes(call, 4, 40000, 4, 8, 2, 128, G.SPMM_BF16)                       # parts of the keys
    assert few > 0 and few % (4 * 8 * 130 * 4) == 0
    assert sizes(call, 0, 0, 1, 1, 1, 1, G.SPMM_F32) == 0
    assert sizes(back, 100, 100, 1, 4, 4, 64, G.SPMM_F32) == 100 * 4 * 4
    long = sizes(back, 8192, 8192, 1, 16, 1, 128, G.SPMM_BF16)                   # parts of the rows
    assert long > 8192 * 16 * 4 and (long - 8192 * 16 * 4) % (2 * 8192 * 128 * 4) == 0
    for name in (call, back):
        assert getattr(G.lib(), name)(1, 1, 1, 1, 1, 1, 0, None) == INV


@pytest.mark.parametrize("call,args", [("spmm_segment_attention", attention), ("spmm_segment_attention_backward", backward)])
def test_attention_sizes_are_refused(call, args):
    for bad in (dict(R=-1), dict(K=-1), dict(S=0), dict(H=0), dict(Hk=0), dict(D=0), dict(H=3, Hk=2), dict(kind=7)):
        refused(INV, call, *args(**bad))
    assert "128" in refused(UNS, call, *args(D=129, ldq=258, ldk=129, ldv=129))
    for bad in (dict(R=BIG), dict(K=BIG), dict(S=2 ** 24), dict(H=2 ** 16, Hk=1), dict(R=2 ** 30, H=2),
                dict(K=2 ** 30, H=4, Hk=2), dict(S=2 ** 23, H=2, Hk=2)):
        refused(UNS, call, *args(**bad))
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-60)):
        assert "scale" in refused(INV, call, *args(**bad))
    for bad in (dict(ldq=15), dict(ldk=7), dict(ldv=0), dict(ldq=BIG)):
        assert "ld" in refused(INV, call, *args(**bad))


def test_attention_arrays_are_refused():
    assert "offsets" in refused(INV, "spmm_segment_attention", *attention())
    assert "workspace" in refused(INV, "spmm_segment_attention", *attention(R=4, K=40000, S=4, D=128, ldq=256, ldk=128, ldv=128))
    assert "all NULL" in refused(INV, "spmm_segment_attention_backward", *backward(dq=n))
    assert "workspace" in refused(INV, "spmm_segment_attention_backward", *backward())
    assert G.lib().spmm_segment_attention(*attention(R=0)) == G.SPMM_OK          # no rows: nothing to do


def test_dropout_is_refused():
    for p in (-0.1, 1.1, float("nan")):
        assert "p must" in refused(INV, "spmm_dropout", n, n, n, 4, p, n, 0, 0, n)
    refused(INV, "spmm_dropout", n, n, n, -1, 0.5, n, 0, 0, n)
    refused(INV, "spmm_dropout", n, n, n, 4, 0.5, n, 0, 9, n)
    refused(UNS, "spmm_dropout", n, n, n, 2 ** 59, 0.5, n, 0, 0, n)
    assert "x is NULL" in refused(INV, "spmm_dropout", n, n, n, 4, 0.5, n, 0, 0, n)
    assert G.lib().spmm_dropout(n, n, n, 0, 0.5, n, 0, 0, n) == G.SPMM_OK


def test_loss_is_refused():
    state, forward, back = sizes("spmm_linear_cross_entropy_workspace", 100, 64, 1000, 0, outputs=3)
    assert state == 100 * 12 + 8 and forward > 0 and back > 100 * 1008 * 4
    # d of all classes of one row would be 2^33 bytes: it is held in pieces
    assert sizes("spmm_linear_cross_entropy_workspace", 1 << 20, 8, 1 << 20, 1, outputs=3)[2] < 1 << 32
    one = ctypes.byref(ctypes.c_int64())
    for bad in ((-1, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (1, 1, 1, 5)):
        refused(INV, "spmm_linear_cross_entropy_workspace", *bad, one, one, one)
    for bad in ((BIG, 1, 1, 0), (1, 2 ** 24, 1, 0), (1, 1, BIG, 0), (2 ** 30, 8, 2 ** 30, 0), (1, 2 ** 23, 2 ** 30, 0)):
        refused(UNS, "spmm_linear_cross_entropy_workspace", *bad, one, one, one)
    assert G.lib().spmm_linear_cross_entropy_workspace(1, 1, 1, 0, None, one, one) == INV
    call = "spmm_linear_cross_entropy"
    assert "reduction" in refused(INV, call, n, n, n, n, 4, 4, 4, 3, 0, n, 0, n, 0, n)
    assert "state" in refused(INV, call, n, n, n, n, 4, 4, 4, 0, 0, n, 0, n, 1 << 20, n)
    assert "workspace" in refused(INV, call, n, n, n, n, 4, 4, 4, 0, 0, n, 1 << 20, n, 0, n)
    assert "x is NULL" in refused(INV, call, n, n, n, n, 4, 4, 4, 0, 0, n, 1 << 20, n, 1 << 20, n)
    call = "spmm_linear_cross_entropy_backward"
    assert "both NULL" in refused(INV, call, n, n, n, n, n, n, 4, 4, 4, 0, 0, n, 0, n, 0, n)
    assert "state" in refused(INV, call, n, n, n, n, 64, n, 4, 4, 4, 0, 0, n, 0, n, 0, n)
    assert "workspace" in refused(INV, call, n, n, n, n, 64, n, 4, 4, 4, 0, 0, n, 1 << 20, n, 0, n)
    assert "x is NULL" in refused(INV, call, n, n, n, n, 64, n, 4, 4, 4, 0, 0, n, 1 << 20, n, 1 << 30, n)


def test_host_tensors_shapes_and_types_are_refused_by_the_binding():
    f, i = torch.zeros, torch.int64
    q, k, o = f(6, 4, 8), f(6, 2, 8), f(3, dtype=i)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.segment_attention(q, k, k, o)
    with pytest.raises(ValueError, match="dimensions"):
        G.segment_attention(f(6, 8), k, k, o)
    with pytest.raises(TypeError, match="one type"):
        G.segment_attention(q, k.half(), k, o)
    with pytest.raises(TypeError, match="float32"):
        G.segment_attention(q.double(), k, k, o)
    x = f(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.dropout(x, 0.5, 1)
    with pytest.raises(TypeError, match="float32"):
        G.dropout(x.to(i), 0.5, 1)
    w, t = f(5, 8), f(4, dtype=i)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.linear_cross_entropy(x, w, t)
    with pytest.raises(TypeError, match="w must be"):
        G.linear_cross_entropy(x, w.half(), t)
    with pytest.raises(ValueError, match="dimensions"):
        G.linear_cross_entropy(f(2, 4, 8), w, t)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.spmm_dropout(x, None, x, 0.5, f(1, dtype=i))
    with pytest.raises(ValueError, match="GPU tensor"):
        G.spmm_segment_attention(q, k, k, o, o, q)
    with pytest.raises(ValueError, match="GPU tensor"):
        G.spmm_linear_cross_entropy(x, w, t, f(()))
