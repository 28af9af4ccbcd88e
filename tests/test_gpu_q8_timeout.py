"""Failure path of the bounded waits of the 8-bit decode and prefill kernels, without faulting the
GPU: the test library (20 ms limits) leaves out one tile of every warp (decode) or one ring unit of
every CTA (prefill), so that a wait runs out; the error is reported, every other load lands, and the
same context then computes the right result."""
import ctypes

import pytest
import torch

from tests.test_gpu_q8 import _case

pytestmark = pytest.mark.gpu

P, I32, I64, F32, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                        ctypes.c_size_t)
ERR_TIMEOUT, DEVERR_TIMEOUT = 4, 8


@pytest.fixture(scope="module")
def test_lib(cuda_lib):
    from paged_kv_cache_09_gb300 import _build
    lib = ctypes.CDLL(_build.build_test())
    lib.pa_test_hook.argtypes = [I32] * 3
    cache = [P, P, P, P, I64, I64, I64]
    lib.pa_decode_q8.argtypes = [P, *cache, P, I64, P] + [I32] * 6 + [F32, P, P, SZ, P]
    lib.pa_prefill_chunk_q8.argtypes = [P, *cache, P] + [I32] * 7 + [F32, P, P, SZ, P]
    lib.pa_get_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint), I32, P]
    assert lib.pa_test_hook(-1, -1, 0) == 0
    yield lib
    lib.pa_test_hook(-1, -1, 0)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _errors(lib):
    v = ctypes.c_uint(0)
    rc = lib.pa_get_device_errors(ctypes.byref(v), 1, _stream())
    return rc, int(v.value)


def _cache(c):
    kc, vc, ks, vs = c["cache"]
    return (kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), kc.stride(0), ks.stride(0),
            kc.shape[0])


@pytest.mark.parametrize("skip", [0, 1, 3])
@pytest.mark.parametrize("lens", [[5000], [300, 0, 2000, 17, 900], [90] * 150])
def test_decode_wait_that_runs_out(test_lib, cuda_lib, lens, skip):
    pa, lib = cuda_lib, test_lib
    c = _case(pa, lens, 64, 24, 4, seed=60)
    S = len(lens)
    ws = torch.empty(pa.decode_q8_workspace_size(S, 24, 4, 256, 64, max(lens)), dtype=torch.uint8,
                     device="cuda")

    def run():
        out = torch.empty_like(c["q"])
        assert lib.pa_decode_q8(
            c["q"].data_ptr(), *_cache(c), c["bt"].data_ptr(), c["bt"].stride(0), c["lens"].data_ptr(),
            S, max(lens), 24, 4, 256, 64, 0.0625, out.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream()) == 0
        return out

    assert _errors(lib) == (0, 0)
    assert lib.pa_test_hook(skip, -1, 0) == 0
    bad = run()
    rc, errs = _errors(lib)
    if skip == 0:  # every warp with any work; later tiles of a warp need not exist
        assert rc == ERR_TIMEOUT and errs == DEVERR_TIMEOUT, (rc, errs)
    assert torch.isfinite(bad.float()).all()
    assert lib.pa_test_hook(-1, -1, 0) == 0
    good = run()
    assert _errors(lib) == (0, 0)
    assert torch.equal(good, pa.decode_q8(c["q"], *c["cache"], c["bt"], c["lens"], 0.0625, max(lens)))
    assert pa.device_errors() == 0


@pytest.mark.parametrize("unit", [0, 2, 7])
@pytest.mark.parametrize("rows,start", [(300, 700), (1, 8000)])
def test_prefill_wait_that_runs_out(test_lib, cuda_lib, rows, start, unit):
    pa, lib = cuda_lib, test_lib
    c = _case(pa, [rows + start], 64, 24, 4, seed=61, rows=rows)
    ws = torch.zeros(pa.prefill_q8_workspace_size(rows, start, True, 24, 4, 256, 64),
                     dtype=torch.uint8, device="cuda")

    def run():
        out = torch.empty_like(c["q"])
        assert lib.pa_prefill_chunk_q8(
            c["q"].data_ptr(), *_cache(c), c["bt"].data_ptr(), rows, start, 1, 24, 4, 256, 64, 0.0625,
            out.data_ptr(), ws.data_ptr(), ws.numel(), _stream()) == 0
        return out

    assert _errors(lib) == (0, 0)
    assert lib.pa_test_hook(-1, unit, 0) == 0
    run()
    rc, errs = _errors(lib)
    if unit < 4:  # any CTA with an item takes at least four units
        assert rc == ERR_TIMEOUT and errs == DEVERR_TIMEOUT, (rc, errs)
    assert lib.pa_test_hook(-1, -1, 0) == 0
    good = run()
    assert _errors(lib) == (0, 0)
    assert torch.equal(good, pa.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], start, True, 0.0625))
    assert pa.device_errors() == 0
