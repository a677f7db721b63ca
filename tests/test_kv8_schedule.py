"""The ragged batches of the GPU tests reach what they are for: a half of a CTA that computes none of
more tiles in a row than the ring of scales holds (8)."""
import pytest

from tests.kv8_schedule import idle_runs, jobs, shares
from tests.test_gpu_kv8_ragged import RAGGED


def test_shares_cover_all_tiles():
    for total, ctas in ((1, 148), (147, 148), (1000, 148), (0, 4)):
        cut = shares(total, ctas)
        assert cut[0][0] == 0 and cut[-1][1] == total and all(a[1] == b[0] for a, b in zip(cut, cut[1:]))


def test_jobs_of_one_sequence():
    # 300 queries over 1,000 tokens, one head each: positions 700 .. 955 and 956 .. 999
    assert jobs([1000], [300], 1, 1, 0) == [(0, 8, [(0, 7), (0, 8)]), (0, 8, [(0, 8), (0, 0)])]
    assert jobs([10], [300], 1, 1, 0)[0] == (0, 1, [(0, 0), (0, 0)])


@pytest.mark.parametrize("lens,new,H,Hkv,D,window", RAGGED)
def test_ragged_batches_leave_halves_idle_for_longer_than_the_ring(lens, new, H, Hkv, D, window):
    assert idle_runs(lens, new, H, Hkv, window) > 2 * 8
