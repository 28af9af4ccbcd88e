"""The compiled module of the short calls beside other threads of the program."""
import ctypes
import importlib.machinery
import importlib.util
import shutil
import subprocess
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

# A library that launches nothing: each call says that it has been entered and then waits, two seconds at
# most, until it is let go; status 77 if it was not.
_WAITING = """
#include <stddef.h>
#include <time.h>
volatile int entered, go;
static int wait_for_go(void) {
    entered = 1;
    for (int i = 0; i < 2000 && !go; ++i) nanosleep(&(struct timespec){0, 1000000}, NULL);
    return go ? 0 : 77;
}
#define CALL(f) int f(void) { return wait_for_go(); }
CALL(pa_reshape_and_cache_q8) CALL(pa_gather_cache_q8) CALL(pa_decode_q8) CALL(pa_prefill_varlen_q8)
CALL(pa_qk_norm_mrope) CALL(pa_qk_norm_mrope_cache)
size_t pa_decode_q8_workspace_size(void) { return 1024; }
size_t pa_prefill_varlen_q8_workspace_size(void) { return 1024; }
"""


@pytest.fixture(scope="module")
def waiting(cuda_lib, tmp_path_factory):
    """(a second copy of the module, over the library that waits; that library)"""
    from paged_kv_cache_09_gb300 import _build
    at = tmp_path_factory.mktemp("bind")
    (at / "waiting.c").write_text(_WAITING)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(at / "waiting.so"), str(at / "waiting.c")], check=True)
    copy = str(at / "pa_bind.so")
    shutil.copy(_build.BIND, copy)
    loader = importlib.machinery.ExtensionFileLoader("pa_bind", copy)
    bind = importlib.util.module_from_spec(importlib.util.spec_from_loader("pa_bind", loader))
    loader.exec_module(bind)
    bind.load(str(at / "waiting.so"))
    return bind, ctypes.CDLL(str(at / "waiting.so"))


@pytest.mark.parametrize("name", ["write_q8", "gather_q8", "decode_q8", "prefill_q8", "mrope", "mrope_cache"])
def test_other_threads_run_while_a_call_waits(cuda_lib, waiting, name):
    # A launch waits while the stream's queue is full.  The lock of the interpreter is free meanwhile: a
    # host function of the stream, or the thread that feeds it, may need it.
    pa = cuda_lib
    bind, lib = waiting
    codes, scales = pa.q8_cache_shapes(2, 16, 1)
    cache = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
    cache[:2] = [c.view(torch.float8_e4m3fn) for c in cache[:2]]
    x = torch.zeros(3, 1, 256, dtype=torch.bfloat16, device="cuda")
    slots, w = torch.arange(3, device="cuda"), x[0, 0].clone()
    table, lens = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    rope = (x, x, w, w, torch.zeros(5, 64, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda"),
            bytes(32), 1e-6, False, 0.0)
    bf = torch.zeros(2, 2, 16, 1, 256, dtype=torch.bfloat16, device="cuda")
    args = {"write_q8": (x, x, *cache, slots), "gather_q8": (*cache, slots),
            "decode_q8": (x, *cache, table, lens, 0.0625, 16, None, None),
            "prefill_q8": (x, *cache, table, [0, 1, 3], [1, 2], True, 0.0625, None, None),
            "mrope": rope, "mrope_cache": (*rope, x, bf[:, 0], bf[:, 1], slots)}[name]
    entered, go = (ctypes.c_int.in_dll(lib, v) for v in ("entered", "go"))
    entered.value = go.value = 0
    torch.cuda.synchronize()

    def let_go():
        while not entered.value:
            pass
        go.value = 1

    thread = threading.Thread(target=let_go)
    thread.start()
    got = getattr(bind, name)(*args)
    entered.value = 1  # (the thread ends whatever the call did)
    thread.join()
    assert got is not None and type(got) is not int  # (a status: it was not let go)


def test_two_threads_on_streams_of_their_own(cuda_lib):
    # Steps of writes, decodes and prefills from two threads at once: the bits of one thread after another.
    pa = cuda_lib
    S, hq, hkv, bs, steps = 4, 8, 2, 16, 60

    def run(seed, stream, out):
        with torch.cuda.stream(stream):
            g = torch.Generator(device="cuda").manual_seed(seed)
            codes, scales = pa.q8_cache_shapes(S * 8, bs, hkv)
            cache = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
            cache[:2] = [c.view(torch.float8_e4m3fn) for c in cache[:2]]
            table = torch.arange(S * 8, dtype=torch.int32, device="cuda").view(S, 8)
            x = torch.randn(steps, 3, S, hq, 256, generator=g, device="cuda").to(torch.bfloat16)
            for i in range(steps):
                q, k, v = x[i, 0], x[i, 1, :, :hkv], x[i, 2, :, :hkv]
                pa.reshape_and_cache_q8(k, v, *cache, torch.arange(S, device="cuda") * 8 * bs + i)
                lens = torch.full((S,), i + 1, dtype=torch.int32, device="cuda")
                out.append(pa.decode_q8(q, *cache, table, lens, 0.0625, steps))
                out.append(pa.prefill_varlen_q8(q, *cache, table, list(range(S + 1)), [i + 1] * S, True, 0.0625))
            out += pa.gather_cache_q8(*cache, torch.arange(steps, device="cuda"))
            stream.synchronize()

    streams = [torch.cuda.Stream() for _ in range(2)]
    want, got = [[], []], [[], []]
    for i in range(2):
        run(i, streams[i], want[i])
    threads = [threading.Thread(target=run, args=(i, streams[i], got[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert len(a) == len(b) == 2 * steps + 2
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert pa.device_errors() == 0
