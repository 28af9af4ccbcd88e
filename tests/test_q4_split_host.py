"""How many places the 4-bit decode's work split puts ahead of a pair's tiles (the function that the
kernel calls, on the host).  CPU only."""
import ctypes
import random
import shutil

import pytest

MOST = 2**31 - 1  # places of all pairs


@pytest.fixture(scope="module")
def lead():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    from paged_kv_cache_09_gb300 import _build
    fn = ctypes.CDLL(_build.build_test()).pa_test_decode_q4_pair_lead
    fn.argtypes, fn.restype = [ctypes.c_uint32, ctypes.c_uint64, ctypes.c_uint32], ctypes.c_int
    return fn


def test_lead_by_hand(lead):
    assert lead(15 * 304, 100, 304) == 0       # shares below 16 tiles
    assert lead(16 * 304, 100, 304) == 8       # half a share
    assert lead(100 * 304, 100, 304) == 16
    assert lead(107, 4, 14) == 0               # one short sequence
    assert lead(8, 8, 1) == 0 and lead(16, 16, 1) == 8


@pytest.mark.parametrize("tiles,pairs", [
    (MOST, 16), (MOST - 200, 16), (MOST, 1 << 32), (MOST // 17 + 1, MOST // 17 + 1),
    (MOST // 2, MOST // 16), (MOST // 2, 1 << 40)])
def test_all_lengths_up_to_the_limit_are_taken(lead, tiles, pairs):
    # What is refused goes by the tiles alone: where the leads do not fit there are none.
    assert lead(tiles, pairs, 304) == 0


def test_places_fit_and_shares_pass_a_lead(lead):
    rng = random.Random(1)
    for _ in range(20000):
        tiles = int(2 ** rng.uniform(0, 31)) - 1 or 1
        pairs = min(tiles, int(2 ** rng.uniform(0, 31)))
        ctas = min(rng.choice([2, 7, 152, 304]), -(-tiles // 8))
        got = lead(tiles, pairs, ctas)
        assert 0 <= got <= 16 and tiles + got * pairs <= MOST and 2 * got <= tiles // ctas
