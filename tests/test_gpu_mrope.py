"""Norm + rotation with positions on several axes, against the plain 64-bit form; and whole serving
steps with it over the 8-bit cache."""
import numpy as np
import pytest
import torch

import _q4
import _q8
from _q4 import f64

pytestmark = pytest.mark.gpu


def _case(T, hq, hkv, dim, rot, n=3, rows=500, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randn(T, (hq + 2 * hkv) * dim, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in packed.split([hq * dim, hkv * dim, hkv * dim], 1))
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, rows, (n, T), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, w, torch.from_numpy(_q4.cos_sin_table(rows, rot)).cuda(), pos


def _ref(x, w, table, pos, axes, interleaved, bias=0.0, eps=1e-6):
    """fp64 rows and the bound: half a BF16 step of the result, and fp32's share of the pair that
    it is made of (a dozen roundings of 2^-24 on values of the row's size)."""
    y = _q8.mrope(f64(x), f64(w), bias, eps, table.double().cpu().numpy(), pos.cpu().numpy(), axes, interleaved)
    plain = _q8.mrope(f64(x), f64(w), bias, eps, np.zeros((1, 0)), pos.cpu().numpy(), [], interleaved)
    big = np.abs(plain).max(-1, keepdims=True)
    return y, np.abs(y) * 2.0 ** -8 * 1.01 + 2.0 ** -19 * big + 1e-30


@pytest.mark.parametrize("dim,rot,hq,hkv,T,interleaved,axes", [
    (256, 64, 24, 4, 16, False, "runs"), (256, 256, 24, 4, 3, False, "turns"), (256, 64, 5, 1, 1, True, "turns"),
    (128, 128, 32, 8, 40, False, "runs"), (128, 32, 6, 2, 7, True, "runs"), (64, 64, 9, 3, 20, False, "turns"),
    (64, 16, 3, 1, 5, True, "random"), (256, 0, 8, 2, 4, False, "runs"), (256, 256, 7, 7, 600, True, "random"),
    (128, 16, 1, 1, 513, False, "random"), (64, 48, 4, 4, 900, False, "turns"),
    (256, 256, 24, 4, 1300, False, "runs"), (64, 64, 15, 5, 2000, True, "runs"), (256, 192, 40, 2, 700, False, "runs"),
])
@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_mrope_matches_plain(cuda_lib, dim, rot, hq, hkv, T, interleaved, axes, n):
    pa = cuda_lib
    q, k, v, w, table, pos = _case(T, hq, hkv, dim, rot, n, seed=n)
    half = rot // 2
    if axes == "random":
        axes = bytes(np.random.default_rng(n).integers(0, n, half).tolist())
    else:
        parts = [half // n] * n
        parts[0] += half - sum(parts)
        axes = pa.mrope_axes(parts, axes == "turns")
    assert len(axes) == half
    qo, ko = pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, interleaved=interleaved)
    for got, x, ww in ((qo, q, w[0]), (ko, k, w[1])):
        ref, tol = _ref(x, ww, table, pos, axes, interleaved)
        assert (np.abs(f64(got) - ref) <= tol).all()
    assert pa.device_errors() == 0


@pytest.mark.parametrize("T,dim,interleaved", [(5, 256, False), (700, 256, True), (33, 128, False), (64, 64, True)])
def test_mrope_of_equal_positions_is_rope(cuda_lib, T, dim, interleaved):
    pa = cuda_lib
    q, k, v, w, table, pos = _case(T, 24, 4, dim, 64, 1, seed=T)
    want = pa.qk_norm_rope(q, k, w[0], w[1], table, pos[0], 1e-6, interleaved=interleaved)
    for turn in (False, True):
        for p in (pos.expand(3, -1).contiguous(), pos.expand(3, -1)):
            got = pa.qk_norm_mrope(q, k, w[0], w[1], table, p, pa.mrope_axes([16, 8, 8], turn), 1e-6,
                                   interleaved=interleaved)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_mrope_padding_range_strides_and_in_place(cuda_lib):
    pa = cuda_lib
    T = 700
    q, k, v, w, table, _ = _case(T, 24, 4, 256, 64, seed=3)
    wide = torch.randint(0, 500, (3, T + 9), device="cuda", dtype=torch.int32)
    pos = wide[:, 4:T + 4]  # rows further apart than tokens
    axes = pa.mrope_axes([16, 8, 8])
    pos[0, 5], pos[1, 6], pos[2, 7] = -1, -1, -9       # padding, on any axis
    pos[0, 8], pos[2, 8] = -1, 500                     # padding all the same
    want_q, want_k = q.clone(), k.clone()
    pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, q_out=want_q, k_out=want_k)
    assert pa.device_errors() == 0
    for a, b in ((want_q, q), (want_k, k)):
        assert torch.equal(a[5:9], b[5:9])
    ref, tol = _ref(q, w[0], table, pos, axes, False)
    live = [t for t in range(T) if not 5 <= t < 9]
    assert (np.abs(f64(want_q) - ref) <= tol)[live].all()
    pos[1, 699] = 500  # past the table
    keep_q, keep_k = want_q.clone(), want_k.clone()
    pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, q_out=want_q, k_out=want_k)
    assert pa.device_errors() == pa.DEVERR_POSITION
    assert torch.equal(want_q, keep_q) and torch.equal(want_k, keep_k)
    pos[1, 699] = 499
    want = pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, weight_bias=1.0)
    plain = v.clone()
    pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, weight_bias=1.0, q_out=q, k_out=k)
    assert torch.equal(q[9:], want[0][9:]) and torch.equal(k[9:], want[1][9:]) and torch.equal(v, plain)


@pytest.mark.parametrize("T,dim,bs,interleaved,turn", [(1, 256, 16, False, True), (16, 256, 832, False, False),
                                                       (600, 256, 64, True, True), (9, 128, 16, False, True),
                                                       (30, 64, 7, True, False)])
def test_mrope_cache_is_the_two_calls(cuda_lib, T, dim, bs, interleaved, turn):
    pa = cuda_lib
    hq, hkv = 12, 4
    q, k, v, w, table, pos = _case(T, hq, hkv, dim, 64, seed=T)
    axes = pa.mrope_axes([16, 8, 8], turn)
    if T > 4:
        pos[1, 3] = -1
    qo, ko = pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6, interleaved=interleaved)
    pages = -(-T // bs) + 1
    slots = torch.randperm(pages * bs, device="cuda")[:T]
    slots[T // 2] = -1
    live = slots.clone()
    if T > 4:
        live[3] = -1
    rows = (pos >= 0).all(0)
    kv = torch.zeros(pages, 2, bs, hkv, dim, dtype=torch.bfloat16, device="cuda")
    want = torch.zeros_like(kv)
    pa.reshape_and_cache(ko, v, want[:, 0], want[:, 1], live)
    got_q = pa.qk_norm_mrope_cache(q, k, v, w[0], w[1], table, pos, axes, 1e-6, kv[:, 0], kv[:, 1], slots,
                                   interleaved=interleaved)
    assert torch.equal(got_q[rows], qo[rows]) and torch.equal(kv, want)
    if dim == 256:
        kc = torch.zeros(pa.q4_cache_shape(pages, bs, hkv), dtype=torch.uint8, device="cuda")
        vc, wk, wv = kc.clone(), kc.clone(), kc.clone()
        pa.reshape_and_cache_q4(ko, v, wk, wv, live)
        got_q = pa.qk_norm_mrope_cache(q, k, v, w[0], w[1], table, pos, axes, 1e-6, kc, vc, slots,
                                       interleaved=interleaved)
        assert torch.equal(got_q[rows], qo[rows]) and torch.equal(kc, wk) and torch.equal(vc, wv)
    assert pa.device_errors() == 0


def test_mrope_refuses(cuda_lib):
    pa = cuda_lib
    q, k, v, w, table, pos = _case(4, 4, 2, 256, 64)
    good = pa.mrope_axes([16, 8, 8])
    for p, axes in ((pos[0], good), (pos[:, :3], good), (pos, good[:-1]),
                    (torch.zeros(5, 4, dtype=torch.int32, device="cuda"), good),
                    (torch.zeros(4, 3, dtype=torch.int32, device="cuda").T, good)):
        with pytest.raises(ValueError):
            pa.qk_norm_mrope(q, k, w[0], w[1], table, p, axes, 1e-6)
    with pytest.raises(pa.PAError):
        pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, bytes(31) + bytes([3]), 1e-6)
    with pytest.raises(pa.PAError):
        pa.qk_norm_mrope(q, k, w[0], w[1], table, pos[:2], good, 1e-6)  # axis 2 of two


@pytest.mark.parametrize("bs", [16, 784])
def test_serving_steps_over_the_q8_cache(cuda_lib, bs):
    """Three requests, one with an image: a mixed step (two prompt chunks and a decode), then decode
    steps, each through prep, norm + rotation, write, and attention; against fp64 over the cache."""
    pa = cuda_lib
    hq, hkv, S, pool = 12, 2, 4, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [(1 + 0.1 * torch.randn(256, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    table = torch.from_numpy(_q4.cos_sin_table(4000, 64)).cuda()
    axes = pa.mrope_axes([12, 10, 10], True)
    codes, scales = pa.q8_cache_shapes(pool, bs, hkv)
    cache = [torch.full(s, 0xFF, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
    cache[:2] = [c.view(torch.float8_e4m3fn) for c in cache[:2]]
    free = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((S, -(-2000 // bs)), -1, dtype=torch.int32, device="cuda")
    computed = torch.zeros(S, dtype=torch.int32, device="cuda")
    plain = [_q8.empty_cache(pool, bs, hkv, 0xFF, 0xFF) for _ in range(2)]
    used = 0
    for step, new in enumerate(([850, 33, 0, 1], [300, 1, 0, 1], [1, 1, 5, 1], [1, 1, 1, 1], [1, 1, 1, 1])):
        T = sum(new)
        prep = pa.batch_input_prep(computed, torch.tensor(new, dtype=torch.int32, device="cuda"), [bt], [bs],
                                   [free[used:]], T)
        used += int(prep["pages_taken"][0])
        packed = torch.randn(T, (hq + 2 * hkv) * 256, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, 256)) for x in packed.split([hq * 256, hkv * 256, hkv * 256], 1))
        p = prep["positions"]
        image = (prep["seq_idx"] == 0) & (p >= 100) & (p < 500)  # 20 x 20 patches
        pos = torch.stack([torch.where(image, 100, p), torch.where(image, 100 + (p - 100) // 20, p),
                           torch.where(image, 100 + (p - 100) % 20, p)]).to(torch.int32)
        qn, kn = pa.qk_norm_mrope(q, k, w[0], w[1], table, pos, axes, 1e-6)
        for got, x, ww in ((qn, q, w[0]), (kn, k, w[1])):
            ref, tol = _ref(x, ww, table, pos, axes, False)
            assert (np.abs(f64(got) - ref) <= tol).all()
        slots = prep["slot_mappings"][0]
        pa.reshape_and_cache_q8(kn, v, *cache, slots)
        for x, c, i in ((kn, plain[0], 0), (v, plain[1], 1)):
            _q8.write(*c, slots.cpu().numpy(), f64(x))
            assert np.array_equal(cache[i].view(torch.uint8).cpu().numpy(), c[0])
            assert np.array_equal(cache[2 + i].cpu().numpy(), c[1])
        cu, lens = prep["query_start_loc"].tolist(), prep["seq_lens"].tolist()
        if max(new) > 1:
            out = pa.prefill_varlen_q8(qn, *cache, bt, cu, lens, True, 0.0625)
            ref, tol = _q8.prefill(f64(qn), *plain, bt.cpu().numpy(), cu, lens, True, 0.0625)
        else:
            out = pa.decode_q8(qn, *cache, bt, prep["seq_lens"], 0.0625, 1400)
            ref, tol = _q8.decode(f64(qn), *plain, bt.cpu().numpy(), lens, 0.0625)
        assert (np.abs(f64(out) - ref) <= tol).all(), step
        computed += torch.tensor(new, dtype=torch.int32, device="cuda")
    assert pa.device_errors() == 0
