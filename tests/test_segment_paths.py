"""The model of the segment product's paths against the library's workspace,
and the paths that the GPU tests' shapes take."""
import ctypes
import random

import pytest

import gnn_sparse_dense_amd as G
from tests.segment_paths import direct, dw_shape, product_tile, slot_of
from tests.test_gpu_segment_paths import DW_CHUNKS, DW_LARGE, PRODUCT


@pytest.mark.parametrize("size,kind", [(4, G.SPMM_F32), (2, G.SPMM_BF16), (2, G.SPMM_F16)])
def test_chunks_of_the_model_are_the_workspace(size, kind):
    n = ctypes.c_int64()
    for R in (0, 1, 4096, 4097, 20011, 150001, 10 ** 6):
        for E in (1, 5, 64, 65, 600):
            for I, O in ((1, 1), (64, 64), (265, 131), (264, 136), (1024, 1024), (2048, 2056)):
                assert G.lib().spmm_segment_workspace(R, E, I, O, kind, ctypes.byref(n)) == G.SPMM_OK
                most = max(dw_shape(R, E, I, O, size, aligned)[3] for aligned in (False, True))
                assert n.value == most * I * O * 4, (R, E, I, O)


def test_shapes_of_the_gpu_tests_reach_their_paths():
    few, many = 0, 0
    for E, I, O in DW_LARGE:
        tile, tiles, chunk, _ = dw_shape(3000, E, I, O, 2)
        assert (tile, chunk) == (256, 0)
        few, many = few + (tiles <= 32), many + (tiles > 32)
    assert few >= 4 and many >= 1
    assert {E > 64 for E, I, O in DW_LARGE} == {False, True}
    chunks = [dw_shape(R, E, I, O, 2) for R, E, I, O in DW_CHUNKS]
    assert all(tile == 128 and chunk > 0 for tile, _, chunk, _ in chunks)
    assert min(c[2] for c in chunks) == 256 < max(c[2] for c in chunks)
    assert max(c[3] for c in chunks) > 64                 # more chunks than one scan covers
    assert {direct(2, I, O) for R, E, I, O in DW_CHUNKS} == {False, True}
    large = [[product_tile(R, I, O, 2, t) for t in (False, True)] for R, E, I, O in PRODUCT]
    for t in (0, 1):
        assert any(p[t][0] == 256 and p[t][1] > 8 for p in large)
        assert {p[t][1] % 4 for p in large if p[t][0] == 256} >= {1, 2, 3}


@pytest.mark.parametrize("E,most", [(1, 900), (63, 700), (64, 20), (300, 90), (4200, 2)])
@pytest.mark.parametrize("length", [128, 256])
def test_every_piece_of_a_run_has_a_slot(E, most, length):
    """Slots of the search against the runs cut one after another."""
    g = random.Random(E + most)
    for empty in ((0.0, 0.5, 1.0) if E < 1000 else (0.5,)):
        bounds = [g.randint(0, 300)]
        for _ in range(E):
            bounds.append(bounds[-1] + (0 if g.random() < empty else g.randint(0, most)))
        R = bounds[-1] + g.choice([0, 1, 500])
        want = [(v, row, hi) for v, (lo, hi) in enumerate(zip([0, *bounds], [*bounds, R])) for row in range(lo, hi, length)]
        slots = [slot_of(bounds, R, length, s) for s in range(R // length + E + 2)]
        assert [s for s in slots if s[1] < s[2]] == want


def test_slots_of_bounds_out_of_order_stay_inside():
    g = random.Random(5)
    for _ in range(30):
        R, E = g.randint(0, 5000), g.randint(1, 200)
        bounds = [g.choice([-7, 0, R, 2 ** 40, g.randint(0, R)]) for _ in range(E + 1)]
        for s in range(R // 128 + E + 2):
            v, row, end = slot_of(bounds, R, 128, s)
            assert 0 <= v <= E + 1 and row >= 0 and end <= R
