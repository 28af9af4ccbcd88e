"""The mixed-step and 4-bit-cache calls: exports, refusals on the host, and the plain
implementations that the GPU tests use, against values worked out by hand.  CPU only."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import _q4

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x10000  # aligned, non-null, never dereferenced on the host
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import shutil
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import paged_kv_cache_09_gb300 as pa
    pa.build()
    return pa.load()


def test_every_declared_call_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pa.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text))
    assert {"pa_batch_input_prep", "pa_qk_norm_rope", "pa_qk_norm_rope_cache", "pa_decode_q4",
            "pa_reshape_and_cache_q4", "pa_gather_cache_q4", "pa_prefill_chunk_q4",
            "pa_prefill_varlen_q4"} <= names
    for n in names:
        assert hasattr(lib, n), n


def _call(fn, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*a.values())


_DEC = dict(q=FAKE, k=FAKE, v=FAKE, page_stride=832 * 4 * 144, num_pages=64, bt=FAKE, bt_stride=16,
            lens=FAKE, num_seqs=1, max_len=8192, hq=24, hkv=4, d=256, bs=832, scale=0.0625, out=FAKE,
            ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(bt=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(num_seqs=0), INVALID), (dict(num_seqs=65536), INVALID), (dict(max_len=0), INVALID),
    (dict(hq=25), INVALID), (dict(hkv=0), INVALID), (dict(bs=0), INVALID),
    (dict(bs=(1 << 20) + 1, page_stride=1 << 40), INVALID),
    (dict(page_stride=832 * 4 * 144 - 16), INVALID), (dict(page_stride=832 * 4 * 144 + 8), INVALID),
    (dict(bt_stride=9), INVALID), (dict(q=FAKE + 8), INVALID), (dict(v=FAKE + 4), INVALID),
    (dict(ws=FAKE + 128), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(num_pages=0), INVALID), (dict(d=128), UNSUPPORTED), (dict(hq=36), UNSUPPORTED),
])
def test_decode_q4_refuses(lib, kw, want):
    assert _call(lib.pa_decode_q4, _DEC, kw) == want


_WRITE = dict(key=FAKE, ks=1024, value=FAKE, vs=1024, k=FAKE, v=FAKE, page_stride=16 * 4 * 144,
              num_pages=8, slots=FAKE, T=5, hkv=4, d=256, bs=16, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(T=0, key=None, k=None), 0), (dict(key=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(ks=1016), INVALID),
    (dict(vs=1028), INVALID), (dict(key=FAKE + 8), INVALID), (dict(d=64), UNSUPPORTED),
    (dict(page_stride=100), INVALID), (dict(k=FAKE + 1), INVALID),
])
def test_write_q4_refuses(lib, kw, want):
    assert _call(lib.pa_reshape_and_cache_q4, _WRITE, kw) == want


_GATHER = dict(k=FAKE, v=FAKE, page_stride=16 * 4 * 144, num_pages=8, slots=FAKE, T=5, hkv=4, d=256,
               bs=16, ko=FAKE, vo=FAKE, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(T=0, ko=None), 0), (dict(ko=None), INVALID),
    (dict(vo=FAKE + 8), INVALID), (dict(d=512), UNSUPPORTED), (dict(num_pages=0), INVALID),
])
def test_gather_q4_refuses(lib, kw, want):
    assert _call(lib.pa_gather_cache_q4, _GATHER, kw) == want


_ROPE = dict(q=FAKE, qs=24 * 256, k=FAKE, ks=1024, v=FAKE, vs=1024, qw=FAKE, kw=FAKE, bias=0.0,
             eps=1e-6, table=FAKE, rows=100, rot=64, il=0, pos=FAKE, T=3, hq=24, hkv=4, d=256,
             qo=FAKE, qos=24 * 256, fmt=0, kc=FAKE, vc=FAKE, page_stride=16 * 1024, num_pages=4,
             slots=FAKE, bs=16, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(qw=None), INVALID),
    (dict(table=None), INVALID), (dict(pos=None), INVALID), (dict(qo=None), INVALID),
    (dict(slots=None), INVALID), (dict(fmt=2), INVALID), (dict(rot=24), INVALID),
    (dict(rot=272), INVALID), (dict(rot=-16), INVALID), (dict(rows=0), INVALID),
    (dict(T=-1), INVALID), (dict(hq=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(qs=24 * 256 - 8), INVALID),
    (dict(ks=1025), INVALID), (dict(kc=FAKE + 8), INVALID), (dict(bs=0), INVALID),
    (dict(page_stride=16 * 1024 - 8), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(d=128, fmt=1), UNSUPPORTED), (dict(T=0, q=None), 0),
])
def test_rope_cache_refuses(lib, kw, want):
    assert _call(lib.pa_qk_norm_rope_cache, _ROPE, kw) == want


def test_rope_refuses(lib):
    a = dict(q=FAKE, qs=24 * 256, k=FAKE, ks=1024, qw=FAKE, kw=FAKE, bias=0.0, eps=1e-6, table=FAKE,
             rows=100, rot=64, il=0, pos=FAKE, T=3, hq=24, hkv=4, d=256, qo=FAKE, qos=24 * 256,
             ko=FAKE, kos=1024, stream=None)
    assert _call(lib.pa_qk_norm_rope, a, dict(ko=None)) == INVALID
    assert _call(lib.pa_qk_norm_rope, a, dict(kos=1000)) == INVALID
    assert _call(lib.pa_qk_norm_rope, a, dict(d=512)) in (INVALID, UNSUPPORTED)


def _prep(lib, S=4, G=2, tables=(FAKE, FAKE), strides=(16, 16), mbs=(10, 10), bss=(832, 16),
          free=(FAKE, FAKE), nfree=(5, 5), T=7, slots=(FAKE, FAKE), computed=FAKE, new=FAKE,
          lens=FAKE, qsl=FAKE, pos=FAKE, own=FAKE):
    arr = lambda t, v: (t * len(v))(*v)
    return lib.pa_batch_input_prep(computed, new, S, G, arr(ctypes.c_void_p, tables),
                                   arr(ctypes.c_int64, strides), arr(ctypes.c_int, mbs),
                                   arr(ctypes.c_int, bss), arr(ctypes.c_void_p, free),
                                   arr(ctypes.c_int, nfree), T, lens, qsl, pos, own,
                                   arr(ctypes.c_void_p, slots), None, None)


@pytest.mark.parametrize("kw", [
    dict(S=-1), dict(T=-1), dict(G=0), dict(tables=(FAKE, None)), dict(strides=(16, 9)),
    dict(mbs=(0, 10)), dict(bss=(832, 0)), dict(nfree=(-1, 5)), dict(free=(None, FAKE)),
    dict(slots=(None, FAKE)), dict(slots=(FAKE + 4, FAKE)), dict(computed=None), dict(new=None),
    dict(lens=None), dict(qsl=None), dict(pos=None), dict(own=None),
    dict(G=9, tables=(FAKE,) * 9, strides=(16,) * 9, mbs=(10,) * 9, bss=(16,) * 9, free=(FAKE,) * 9,
         nfree=(5,) * 9, slots=(FAKE,) * 9),
])
def test_batch_prep_refuses(lib, kw):
    assert _prep(lib, **kw) == INVALID


def _varlen(lib, cu=(0, 10, 30), lens=(10, 40), bt_stride=1, B=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, page_stride=832 * 4 * 144, num_pages=64, bt=FAKE, hq=24, hkv=4,
             d=256, bs=832, scale=0.0625, out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.pa_prefill_varlen_q4(
        a["q"], a["k"], a["v"], a["page_stride"], a["num_pages"], a["bt"], bt_stride,
        (ctypes.c_int32 * len(cu))(*cu), (ctypes.c_int32 * max(1, len(lens)))(*lens),
        len(lens) if B is None else B, 1, a["hq"], a["hkv"], a["d"], a["bs"], a["scale"], a["out"],
        a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cu=(1, 10, 30)), INVALID), (dict(cu=(0, 10, 5)), INVALID), (dict(lens=(5, 40)), INVALID),
    (dict(lens=(10, 900)), INVALID), (dict(q=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws=FAKE + 16), INVALID), (dict(scale=float("nan")), INVALID), (dict(d=128), UNSUPPORTED),
    (dict(hq=36), UNSUPPORTED), (dict(hq=25), INVALID), (dict(page_stride=8), INVALID),
    (dict(B=-1), INVALID), (dict(cu=(0, 0, 0), q=None, ws=None), 0),
    (dict(cu=(0,), lens=(), B=0, q=None), 0),
])
def test_prefill_q4_refuses(lib, kw, want):
    assert _varlen(lib, **kw) == want


def test_workspace_sizes_of_bad_shapes_are_zero(lib):
    assert lib.pa_decode_q4_workspace_size(0, 24, 4, 256, 832, 8192) == 0
    assert lib.pa_decode_q4_workspace_size(1, 24, 4, 128, 832, 8192) == 0
    assert lib.pa_prefill_q4_workspace_size(0, 0, 1, 24, 4, 256, 832) == 0
    assert lib.pa_prefill_q4_workspace_size(1, 2**31 - 1, 1, 24, 4, 256, 832) == 0


def test_python_refuses_host_tensors():
    import paged_kv_cache_09_gb300 as pa
    with pytest.raises(TypeError):
        pa.reshape_and_cache_q4(torch.zeros(1, 1, 256, dtype=torch.bfloat16),
                                torch.zeros(1, 1, 256, dtype=torch.bfloat16),
                                torch.zeros(pa.q4_cache_shape(1, 16, 1), dtype=torch.uint8),
                                torch.zeros(pa.q4_cache_shape(1, 16, 1), dtype=torch.uint8),
                                torch.zeros(1, dtype=torch.int64))


# ---- the plain implementations
def test_plain_quantiser_by_hand():
    x = np.zeros((1, 256))
    x[0, 64:128] = np.arange(64) % 16          # step 1, codes 0..15
    x[0, 128:192] = 5.0                        # equal values: step 0, kept
    x[0, 192:] = np.where(np.arange(64) % 2, 1.0, -2.0)  # range 3: step 0.2 in BF16
    n, s, lo = _q4.quantise(x)
    assert s[0].tolist()[:3] == [0.0, 1.0, 0.0] and lo[0].tolist() == [0.0, 0.0, 5.0, -2.0]
    assert s[0, 3] == 0.2001953125 and n[0, 192:194].tolist() == [0, 15]
    assert n[0, 64:80].tolist() == list(range(16))
    v = _q4.value(n, s, lo)
    assert np.array_equal(v[0, :192], x[0, :192])
    # ties go to even codes: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    x[0, 64:128] = 0
    x[0, 64:69] = [15, 0.5, 1.5, 2.5, 0]
    n, _, _ = _q4.quantise(x)
    assert n[0, 64:69].tolist() == [15, 0, 2, 2, 0]


def test_plain_layout_by_hand():
    cache = _q4.empty_cache(2, 3, 2, fill=0)
    n = np.zeros(256, np.int64)
    n[64 + 8 * 5 + 3] = 9  # group 1, unit 5, code 3
    _q4.store(cache, 3, 1 * 3 + 2, 1, n, np.array([1.0, 0, 0, 0]), np.array([0, 0, 0, -2.0]))
    run = cache[1, 1]
    assert run[2 * 128 + (5 ^ 2) * 16 + 4 + 1] == 0x90
    assert run[3 * 128 + 2 * 16:3 * 128 + 3 * 16].tolist() == [0x80, 0x3F] + [0] * 12 + [0x00, 0xC0]
    assert int((cache != 0).sum()) == 4
    v, s = _q4.load(cache, 3, np.array([1]), np.array([2]), 1)
    assert v[0, 192:].tolist() == [-2.0] * 64 and s[0].tolist() == [1, 0, 0, 0]


def test_plain_batch_prep_by_hand():
    table = np.array([[7, -1, -1], [3, -1, -1], [4, 5, -1]], np.int32)
    got, short = _q4.batch_prep(np.array([3, 4, 7]), np.array([6, 0, 2]), [table], [4],
                                [np.array([20, 21, 22], np.int32)], 10)
    assert got["seq_lens"].tolist() == [9, 0, 9] and got["query_start_loc"].tolist() == [0, 6, 6, 8]
    assert got["tables"][0].tolist() == [[7, 20, 21], [3, -1, -1], [4, 5, 22]]
    assert got["positions"].tolist() == [3, 4, 5, 6, 7, 8, 7, 8, -1, -1]
    assert got["seq_idx"].tolist() == [0] * 6 + [2, 2, -1, -1]
    assert got["slot_mappings"][0].tolist() == [31, 80, 81, 82, 83, 84, 23, 88, -1, -1]
    assert got["pages_taken"].tolist() == [3] and not short


def test_plain_attention_and_rope_by_hand():
    o = _q4.attend(np.zeros((2, 256)), np.ones((3, 256)), np.arange(3.0)[:, None] * np.ones(256), 1.0,
                   [1, 3])
    assert np.allclose(o[:, 0], [0.0, 1.0])
    table = np.array([[1.0, 0.0], [0.0, 1.0]], np.float32)  # a quarter turn at position 1
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y = _q4.rope(x, np.ones(4), 0.0, 0.0, table, [1], True)
    assert np.allclose(y[0, 0], np.array([-4.0, 3.0, 0, 0]) / 2.5)
