"""The calls of the 8-bit cache and of rotation by several axes: refusals on the host, and the plain
implementations that the GPU tests use, against torch's conversion and values worked out by hand.
CPU only."""
import ctypes
import shutil

import numpy as np
import pytest
import torch

import _q8

INVALID, UNSUPPORTED = 1, 2
FAKE = 0x10000  # aligned, non-null, never dereferenced on the host
PAGE, SCALES = 832 * 4 * 256, 52 * 4


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    import paged_kv_cache_09_gb300 as pa
    pa.build()
    return pa.load()


def _call(fn, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*a.values())


_CACHE = [(dict(k=None), INVALID), (dict(vs=None), INVALID), (dict(k=FAKE + 8), INVALID),
          (dict(page_stride=PAGE - 16), INVALID), (dict(page_stride=PAGE + 8), INVALID),
          (dict(page_stride=1 << 40), INVALID), (dict(scale_stride=SCALES - 1), INVALID),
          (dict(scale_stride=PAGE + 1), INVALID), (dict(num_pages=0), INVALID), (dict(bs=0), INVALID),
          (dict(bs=(1 << 20) + 1, page_stride=1 << 39, scale_stride=1 << 30), INVALID),
          (dict(hkv=0), INVALID), (dict(d=128), UNSUPPORTED)]

_WRITE = dict(key=FAKE, kst=1024, value=FAKE, vst=1024, k=FAKE, v=2 * FAKE, ks=FAKE, vs=FAKE + 3,
              page_stride=PAGE, scale_stride=SCALES, num_pages=8, slots=FAKE, T=5, hkv=4, d=256, bs=832,
              stream=None)


@pytest.mark.parametrize("kw,want", _CACHE + [
    (dict(T=-1), INVALID), (dict(T=0, key=None, k=None), 0), (dict(key=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(kst=1016), INVALID),
    (dict(vst=1028), INVALID), (dict(key=FAKE + 8), INVALID), (dict(v=FAKE), INVALID), (dict(vs=FAKE), INVALID)])
def test_write_q8_refuses(lib, kw, want):
    assert _call(lib.pa_reshape_and_cache_q8, _WRITE, kw) == want


_GATHER = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, page_stride=PAGE, scale_stride=SCALES, num_pages=8,
               slots=FAKE, T=5, hkv=4, d=256, bs=832, ko=FAKE, vo=FAKE, stream=None)


@pytest.mark.parametrize("kw,want", _CACHE + [
    (dict(T=-1), INVALID), (dict(T=0, ko=None), 0), (dict(ko=None), INVALID),
    (dict(vo=FAKE + 8), INVALID), (dict(slots=None), INVALID)])
def test_gather_q8_refuses(lib, kw, want):
    assert _call(lib.pa_gather_cache_q8, _GATHER, kw) == want


_DEC = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, page_stride=PAGE, scale_stride=SCALES, num_pages=64,
            bt=FAKE, bt_stride=16, lens=FAKE, num_seqs=1, max_len=8192, hq=24, hkv=4, d=256, bs=832,
            scale=0.0625, out=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,want", _CACHE + [
    (dict(q=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(num_seqs=0), INVALID),
    (dict(num_seqs=65536), INVALID), (dict(max_len=0), INVALID), (dict(hq=25), INVALID),
    (dict(bt_stride=9), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 4), INVALID),
    (dict(ws=FAKE + 128), INVALID), (dict(scale=float("inf")), INVALID), (dict(hq=36), UNSUPPORTED)])
def test_decode_q8_refuses(lib, kw, want):
    assert _call(lib.pa_decode_q8, _DEC, kw) == want


def _i32(*x):
    return ctypes.cast((ctypes.c_int32 * len(x))(*x), ctypes.c_void_p)


_PRE = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, page_stride=PAGE, scale_stride=SCALES, num_pages=64,
            bt=FAKE, bt_stride=16, cu=_i32(0, 5), lens=_i32(100), num_seqs=1, causal=1, hq=24, hkv=4,
            d=256, bs=832, scale=0.0625, out=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", _CACHE + [
    (dict(q=None), INVALID), (dict(bt=None), INVALID), (dict(ws=None), INVALID), (dict(cu=None), INVALID),
    (dict(lens=_i32(4)), INVALID), (dict(cu=_i32(1, 5)), INVALID), (dict(lens=_i32(16 * 832 + 1)), INVALID),
    (dict(ws=FAKE + 64), INVALID), (dict(hq=25), INVALID), (dict(hq=36), UNSUPPORTED),
    (dict(num_seqs=0), 0)])
def test_prefill_q8_refuses(lib, kw, want):
    assert _call(lib.pa_prefill_varlen_q8, _PRE, kw) == want


_ROPE = dict(q=FAKE, qs=24 * 256, k=FAKE, ks=1024, v=FAKE, vs=1024, qw=FAKE, kw=FAKE, bias=0.0,
             eps=1e-6, table=FAKE, rows=100, rot=64, il=0, pos=FAKE, pos_stride=3, n=3, axes=bytes(32), T=3,
             hq=24, hkv=4, d=256, qo=FAKE, qos=24 * 256, fmt=0, kc=FAKE, vc=FAKE, page_stride=16 * 1024,
             num_pages=4, slots=FAKE, bs=16, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), INVALID), (dict(n=5), INVALID), (dict(axes=None), INVALID), (dict(pos_stride=-1), INVALID),
    (dict(axes=bytes(31) + b"\x03"), INVALID), (dict(axes=b"\xff" + bytes(31)), INVALID),
    (dict(q=None), INVALID), (dict(v=None), INVALID), (dict(table=None), INVALID), (dict(pos=None), INVALID),
    (dict(fmt=2), INVALID), (dict(rot=24), INVALID), (dict(rot=272, axes=bytes(136)), INVALID),
    (dict(rot=-16), INVALID), (dict(rows=0), INVALID), (dict(T=-1), INVALID), (dict(kc=FAKE + 8), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=128, fmt=1), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
    (dict(T=0, q=None), 0)])
def test_mrope_cache_refuses(lib, kw, want):
    assert _call(lib.pa_qk_norm_mrope_cache, _ROPE, kw) == want


def test_lengths_past_32_bits_are_refused(lib):
    import paged_kv_cache_09_gb300 as pa
    past = 2**32
    with pytest.raises(ValueError):
        pa.prefill_varlen_q8_workspace_size([0, 10], [past + 10], True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.prefill_q8_workspace_size(10, past, True, 24, 4, 256, 832)
    with pytest.raises(ValueError):
        pa.decode_q8_workspace_size(1, 24, 4, 256, 832, past + 100)


def test_calls_refuse_what_is_no_cuda_tensor(lib):
    import paged_kv_cache_09_gb300 as pa
    codes, scales = pa.q8_cache_shapes(1, 16, 1)
    kc, ks = torch.zeros(codes, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(scales, dtype=torch.uint8)
    q, bt = torch.zeros(3, 6, 256, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError):
        pa.decode_q8(q, kc, kc, ks, ks, bt, bt[0], 0.0625, 16)
    with pytest.raises(TypeError):
        pa.prefill_chunk_q8(q, kc, kc, ks, ks, bt, 0, True, 0.0625)
    with pytest.raises(TypeError):
        pa.reshape_and_cache_q8(q, q, kc, kc, ks, ks, bt[0])
    with pytest.raises(TypeError):
        pa.gather_cache_q8(kc, kc, ks, ks, bt[0])


def test_short_calls_leave_the_unusual_to_python(lib):
    import paged_kv_cache_09_gb300 as pa
    assert pa._bind is not None
    t = torch.zeros(3, 6, 256, dtype=torch.bfloat16)
    for name, n in (("write_q8", 7), ("gather_q8", 5), ("decode_q8", 11), ("prefill_q8", 12), ("mrope", 10), ("mrope_cache", 14)):
        f = getattr(pa._bind, name)
        for args in ([], [None] * n, [t] * n, [t] * (n + 1), [3] * n, ["x"] * n):
            assert f(*args) is None
    with pytest.raises(RuntimeError):
        pa._bind.load("/nowhere/libpa.so")


def test_axes_of_sections(lib):
    import paged_kv_cache_09_gb300 as pa
    assert list(pa.mrope_axes([3, 2, 1])) == [0, 0, 0, 1, 1, 2]
    assert list(pa.mrope_axes([4, 2, 2], True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(pa.mrope_axes([8])) == [0] * 8
    assert sorted(pa.mrope_axes([12, 10, 10], True)) == [0] * 12 + [1] * 10 + [2] * 10
    assert pa.q8_cache_shapes(3, 20, 2) == ((3, 20, 2, 256), (3, 2, 2))


# ------------------------------------------------------------------------------ the plain forms
def test_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = _q8.decoded(codes.numpy())
    assert np.array_equal(got, want, equal_nan=True)
    x = torch.cat([torch.randn(4000) * s for s in (1e-3, 0.02, 1.0, 100.0)]).clamp(-448, 448)
    mid = (torch.from_numpy(_q8._POSITIVE[1:]) + torch.from_numpy(_q8._POSITIVE[:-1])).float() / 2
    x = torch.cat([x, mid, -mid, torch.tensor([0.0, -0.0, 448.0, -448.0])])
    assert np.array_equal(_q8.encoded(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("top,byte", [(0.0, 1), (448.0, 127), (448.0001, 128), (1.0, 119), (0.875, 118),
                                      (0.876, 119), (2.0 ** -133, 1), (3.3895e38, 247)])
def test_scale_byte(top, byte):
    assert _q8.scale_byte(top) == byte


def test_write_by_hand():
    codes, scales = _q8.empty_cache(1, 20, 1, fill=0x38, scale=127)  # ones
    x = np.zeros((2, 1, 256))
    x[0, 0, :3] = 500, -3, 0.3                # byte 128: 250, -1.5, .15
    x[1, 0, 0] = 2.0 ** -9
    _q8.write(codes, scales, [5, 17], x)
    assert scales[0, :, 0].tolist() == [128, 127]   # the second block stays: nothing larger
    assert (codes[0, :5, 0] == 0x30).all() and (codes[0, 6:16, 0] == 0x30).all()  # a half
    assert _q8.decoded(codes[0, 5, 0, :3]).tolist() == [256.0, -1.5, 0.15625]
    assert codes[0, 17, 0, 0] == 1 and (codes[0, 16, 0] == 0x38).all()
    _q8.write(codes, scales, [0, 3, 3], np.stack([x[1], x[0], x[1]]))  # begins the first block anew
    assert scales[0, 0, 0] == 110 and codes[0, 0, 0, 0] == codes[0, 3, 0, 0] == 0x78  # 256 2^-17
    assert (codes[0, 4, 0] == 0x30).all()


def test_bound_takes_the_kernels_rounding_and_refuses_a_missing_tile():
    rng = np.random.default_rng(1)
    N = 1701
    q, k, v = rng.standard_normal((1, 256)), rng.standard_normal((N, 256)), rng.standard_normal((N, 256))
    ref, tol = _q8.attend(q, k, v, 0.0625, [N])
    x = (k @ q[0]) * 0.0625
    w = (np.exp(x - x.max()) * 64).astype(np.float16).astype(np.float64)
    l = np.exp(x - x.max()).sum() * 64
    got = torch.from_numpy((w @ v) / l).to(torch.bfloat16).double().numpy()
    assert (np.abs(got - ref[0]) <= tol[0]).all()
    for t in range(0, N, 16):
        keep = np.ones(N, bool)
        keep[t:t + 16] = False
        assert not (np.abs((w[keep] @ v[keep]) / w[keep].sum() - ref[0]) <= tol[0]).all(), t
