"""Row operators, without a GPU: sizes, types and arrays that are refused
before the device is touched, and the workspace calls."""
import ctypes

import pytest
import torch

import gnn_sparse_dense_amd as G

BIG = 2 ** 31


def refused(status, call, *args):
    assert getattr(G.lib(), call)(*args) == status, G.spmm_last_error()
    return G.spmm_last_error()[1]


def bytes_of(call, *sizes):
    n = ctypes.c_int64(-1)
    assert getattr(G.lib(), call)(*sizes, ctypes.byref(n)) == G.SPMM_OK, G.spmm_last_error()
    return n.value


def test_workspaces():
    assert bytes_of("spmm_route_workspace", 0, 8) == 0
    assert bytes_of("spmm_route_workspace", 4096, 511) == 0          # one block holds it
    assert bytes_of("spmm_route_workspace", 4097, 511) > 0
    assert bytes_of("spmm_route_workspace", 0, 2048) > 0
    assert bytes_of("spmm_segment_workspace", 0, 4, 8, 8, G.SPMM_BF16) == 0
    assert bytes_of("spmm_segment_workspace", 10 ** 6, 4, 64, 64, G.SPMM_F32) % (4 * 4 * 64 * 64) == 0
    assert bytes_of("spmm_layer_norm_workspace", 0, 64, G.SPMM_F32) >= 2 * 64 * 4
    assert bytes_of("spmm_layer_norm_workspace", 10 ** 6, 10 ** 5, G.SPMM_F16) % (2 * 10 ** 5 * 4) == 0
    for call, sizes in (("spmm_route_workspace", (1, 1)), ("spmm_segment_workspace", (1, 1, 1, 1, 0)),
                        ("spmm_layer_norm_workspace", (1, 1, 0))):
        assert getattr(G.lib(), call)(*sizes, None) == G.SPMM_E_INVALID_ARG


def test_sizes_and_types_are_refused_by_the_library():
    inv, uns = G.SPMM_E_INVALID_ARG, G.SPMM_E_UNSUPPORTED
    one = ctypes.byref(ctypes.c_int64())
    refused(inv, "spmm_route_workspace", -1, 4, one)
    refused(inv, "spmm_route_workspace", 4, 0, one)
    refused(uns, "spmm_route_workspace", BIG, 4, one)
    assert "2048" in refused(uns, "spmm_route_workspace", 4, 2049, one)
    n = None
    assert "expert" in refused(inv, "spmm_route_build", n, 4, 4, n, n, n, n, 0, n)
    assert "workspace" in refused(inv, "spmm_route_build", n, 10 ** 6, 4, n, n, n, n, 16, n)
    for call, rest in (("spmm_route_dispatch", (n, 8, 0, n)), ("spmm_route_combine", (n, 8, 0, n))):
        refused(inv, call, n, n, -1, 2, 4, n, n, 0, *rest)
        refused(inv, call, n, n, 4, 0, 4, n, n, 0, *rest)
        refused(inv, call, n, n, 4, 2, 0, n, n, 0, *rest)
        refused(uns, call, n, n, BIG, 2, 4, n, n, 0, *rest)
        refused(uns, call, n, n, BIG // 2, 2, 4, n, n, 0, *rest)
        assert "N" in refused(inv, call, n, n, 4, 2, 4, n, n, 0, n, 0, 0, n)
        assert "type" in refused(inv, call, n, n, 4, 2, 4, n, n, 0, n, 8, 3, n)
        assert "fp32 or" in refused(inv, call, n, n, 4, 2, 4, n, 64, G.SPMM_F16, n, 8, G.SPMM_BF16, n)
        assert "offsets" in refused(inv, call, n, n, 4, 2, 4, n, n, 0, *rest)
    assert "both NULL" in refused(inv, "spmm_route_combine_backward", n, n, 4, 2, 4, n, n, 0, n, n, n, 8, 0, n)
    for call in ("spmm_segment_product", "spmm_segment_product_dx"):
        refused(inv, call, n, n, n, n, -1, 1, 1, 1, 0, n)
        refused(inv, call, n, n, n, n, 4, 1, 1, 1, 0, n)
        refused(inv, call, n, n, n, n, 0, 0, 1, 1, 0, n)
        refused(inv, call, n, n, n, n, 0, 1, 1, 0, 0, n)
        refused(inv, call, n, n, n, n, 0, 1, 1, 1, 7, n)
        refused(uns, call, n, n, n, n, 0, 1, 2 ** 24, 1, 0, n)
        refused(uns, call, n, n, n, n, 0, 2 ** 23, 2 ** 23, 2 ** 23, 0, n)
        assert getattr(G.lib(), call)(n, n, n, n, 0, 1, 1, 1, 0, n) == G.SPMM_OK      # no rows: nothing to do
    assert "workspace" in refused(inv, "spmm_segment_product_dw", 64, 64, n, n, 10 ** 6, 4, 64, 64, 0, n, 0, n)
    refused(inv, "spmm_layer_norm", n, n, n, 0, n, n, n, 4, 0, 1e-5, 0, n)
    refused(inv, "spmm_layer_norm", n, n, n, 0, n, n, n, -4, 8, 1e-5, 0, n)
    refused(uns, "spmm_layer_norm", n, n, n, 0, n, n, n, BIG - 2, BIG - 2, 1e-5, 0, n)
    assert "eps" in refused(inv, "spmm_layer_norm", n, n, n, 0, n, n, n, 4, 8, -1.0, 0, n)
    assert "eps" in refused(inv, "spmm_layer_norm", n, n, n, 0, n, n, n, 4, 8, float("nan"), 0, n)
    assert "together" in refused(inv, "spmm_layer_norm", n, n, n, 0, n, 64, n, 4, 8, 1e-5, 0, n)
    assert "x is NULL" in refused(inv, "spmm_layer_norm", n, n, n, 0, n, n, n, 4, 8, 1e-5, 0, n)
    assert "all NULL" in refused(inv, "spmm_layer_norm_backward", n, n, n, 0, n, n, n, n, n, 4, 8, 0, n, 0, n)
    assert "workspace" in refused(inv, "spmm_layer_norm_backward", n, n, n, 0, n, n, n, 64, n, 4, 8, 0, n, 0, n)


def test_host_tensors_shapes_and_types_are_refused_by_the_binding():
    i64 = torch.int64
    with pytest.raises(ValueError, match="GPU"):
        G.RowRoute(torch.zeros((4, 2), dtype=i64), 3)
    with pytest.raises(TypeError, match="int64"):
        G.RowRoute(torch.zeros((4, 2), dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="dimensions"):
        G.RowRoute(torch.zeros((4, 2, 1), dtype=i64), 3)
    x, w, o = torch.zeros(4, 8), torch.zeros(2, 8, 5), torch.zeros(3, dtype=i64)
    with pytest.raises(ValueError, match="GPU"):
        G.segment_matmul(x, w, o)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        G.segment_matmul(x.double(), w, o)
    with pytest.raises(TypeError, match="w must be float32"):
        G.segment_matmul(x, w.half(), o)
    with pytest.raises(ValueError, match="dimensions"):
        G.segment_matmul(x, w[0], o)
    with pytest.raises(ValueError, match="GPU"):
        G.layer_norm(x)
    with pytest.raises(TypeError, match="weight must be"):
        G.layer_norm(x, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="shape"):
        G.layer_norm(x, torch.zeros(7))


class FakeRoute:
    T, k, E, device = 4, 2, 3, torch.device("cpu")
    offsets = order = position = torch.zeros(4, dtype=torch.int64)


def test_shapes_of_the_exchange_are_refused_by_the_binding():
    r = FakeRoute()
    with pytest.raises(ValueError, match=r"x has shape \(5, 8\), expected \(4, 8\)"):
        G.dispatch(r, torch.zeros(5, 8))
    with pytest.raises(TypeError, match="float32"):
        G.dispatch(r, torch.zeros(4, 8, dtype=torch.int64))
    with pytest.raises(ValueError, match=r"rows has shape \(4, 8\), expected \(8, 8\)"):
        G.combine(r, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="GPU"):
        G.combine(r, torch.zeros(8, 8))
