"""Attention of batches whose segments differ much in length, against 64 bits
(tests/rows64.py): the launches go by the mean length, so a long segment among many
short ones is walked by tiles and parts that were chosen for the short ones."""
import pytest

pytestmark = pytest.mark.gpu

from tests.test_gpu_attention import compare  # noqa: E402
from tests.test_gpu_rows import TYPES  # noqa: E402


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("place", ["first", "inside", "last"])
def test_single_rows_of_sequences_of_uneven_lengths(place, kind):
    keys = [5, 1, 0, 17] * 12
    keys.insert({"first": 0, "inside": 20, "last": len(keys)}[place], 7000)
    compare([1] * len(keys), keys, 8, 2, 64, kind, True)
    compare([1] * 3, [400, 9000, 300], 4, 2, 128, kind, False, back=2)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("causal", [False, True])
def test_one_long_segment_among_short_ones(causal, kind):
    rows = [6, 1, 0, 11] * 60
    rows.insert(100, 1300)
    compare(rows, None, 2, 1, 32, kind, causal)
    compare(rows, [n // 2 for n in rows], 2, 2, 40, kind, causal, front=1)
    compare([4] * 50 + [3], [2] * 50 + [2500], 2, 1, 96, kind, causal)
