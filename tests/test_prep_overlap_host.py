"""pa_batch_input_prep refuses outputs over its inputs, on the host.  CPU only."""
import ctypes
import shutil

import pytest

OK, INVALID, CUDA = 0, 1, 3


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    import paged_kv_cache_09_gb300 as pa
    pa.build()
    return pa.load()


_AT = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ["computed", "new", "lens", "qsl", "pos", "own", "taken", "table0", "table1", "free0", "free1", "slot0", "slot1"])}


def _prep(lib, S=8, T=20, width=10, stride=10, **at):
    a = dict(_AT, **at)
    two = lambda t, x, y: (t * 2)(x, y)
    P, I = ctypes.c_void_p, ctypes.c_int
    return lib.pa_batch_input_prep(
        a["computed"], a["new"], S, 2, two(P, a["table0"], a["table1"]), two(ctypes.c_int64, stride, stride),
        two(I, width, width), two(I, 16, 832), two(P, a["free0"], a["free1"]), two(I, 50, 50), T, a["lens"],
        a["qsl"], a["pos"], a["own"], two(P, a["slot0"], a["slot1"]), a["taken"], None)


@pytest.mark.parametrize("kw", [
    dict(lens=_AT["computed"]), dict(lens=_AT["new"]), dict(lens=_AT["computed"] + 28),
    dict(lens=_AT["computed"] - 28), dict(qsl=_AT["new"]), dict(pos=_AT["computed"] - 76),
    dict(own=_AT["new"]), dict(taken=_AT["computed"] + 4), dict(slot1=_AT["new"]), dict(lens=_AT["free1"]),
    dict(pos=_AT["table0"]), dict(slot0=_AT["table1"]), dict(table0=_AT["computed"]), dict(table1=_AT["free0"]),
    dict(table0=_AT["table1"]), dict(taken=_AT["free0"] + 196)])
def test_overlaps_are_refused(lib, kw):
    assert _prep(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(), dict(lens=_AT["computed"] + 32), dict(lens=_AT["computed"] - 32), dict(free1=_AT["free0"]),
    dict(taken=None), dict(table1=_AT["table0"] + 40, stride=20), dict(S=0, table0=None, table1=None),
    dict(T=0, slot0=_AT["new"])])
def test_neighbours_and_shared_free_lists_are_taken(lib, kw):
    # (past the arguments: no device here)
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert _prep(lib, **kw) == CUDA
