"""Rotation of calls with many heads: KV heads that take a token's warps more than one round, whose rows
are not copied ahead, and query heads at the ends of what a token's CTAs take."""
import numpy as np
import pytest
import torch

from _q4 import f64
from test_gpu_mrope import _case, _ref

pytestmark = pytest.mark.gpu


# A large call has 4 * 256 / dim rows a round and CTA, and one CTA a token up to 24 * 256 / dim query heads.
@pytest.mark.parametrize("T,hq,hkv,dim", [(600, 12, 9, 256), (500, 30, 30, 256), (700, 8, 17, 128), (900, 5, 40, 64),
                                          (1300, 24, 24, 128)])
@pytest.mark.parametrize("interleaved,turn,one", [(False, False, False), (True, True, False), (False, True, False),
                                                  (False, False, True)])
def test_many_kv_heads(cuda_lib, T, hq, hkv, dim, interleaved, turn, one):
    pa = cuda_lib
    q, k, v, w, table, pos = _case(T, hq, hkv, dim, 64, seed=T)
    axes = pa.mrope_axes([16, 8, 8], turn)
    pos[1, 3] = -1
    if one:  # one position a token
        pos = pos[1:2].expand(3, -1).contiguous()
        how, args = (pa.qk_norm_rope, pa.qk_norm_rope_cache), (table, pos[0], 1e-6)
    else:
        how, args = (pa.qk_norm_mrope, pa.qk_norm_mrope_cache), (table, pos, axes, 1e-6)
    qo, ko = how[0](q, k, *w, *args, interleaved=interleaved)
    rows = (pos >= 0).all(0)
    keep = rows.cpu().numpy()
    for got, x, ww in ((qo, q, w[0]), (ko, k, w[1])):
        ref, tol = _ref(x, ww, table, pos, axes, interleaved)
        assert (np.abs(f64(got) - ref) <= tol)[keep].all()
    bs = 64
    pages = -(-T // bs) + 1
    slots = torch.randperm(pages * bs, device="cuda")[:T]
    slots[T // 2] = -1
    live = torch.where(rows, slots, -1)
    kv = torch.zeros(pages, 2, bs, hkv, dim, dtype=torch.bfloat16, device="cuda")
    want = torch.zeros_like(kv)
    pa.reshape_and_cache(ko, v, want[:, 0], want[:, 1], live)
    got = how[1](q, k, v, *w, *args, kv[:, 0], kv[:, 1], slots, interleaved=interleaved)
    assert torch.equal(got[rows], qo[rows]) and torch.equal(kv, want)
    if dim == 256:
        kc = torch.zeros(pa.q4_cache_shape(pages, bs, hkv), dtype=torch.uint8, device="cuda")
        vc, wk, wv = kc.clone(), kc.clone(), kc.clone()
        pa.reshape_and_cache_q4(ko, v, wk, wv, live)
        got = how[1](q, k, v, *w, *args, kc, vc, slots, interleaved=interleaved)
        assert torch.equal(got[rows], qo[rows]) and torch.equal(kc, wk) and torch.equal(vc, wv)
    assert pa.device_errors() == 0


# 24 * 256 / dim query heads a CTA in a large call, one a warp in a small one.
@pytest.mark.parametrize("hq,hkv,dim", [(24, 1, 256), (25, 1, 256), (49, 7, 256), (48, 2, 128), (97, 1, 128), (96, 3, 64),
                                        (193, 1, 64)])
@pytest.mark.parametrize("T", [2, 620])
def test_many_query_heads(cuda_lib, T, hq, hkv, dim):
    pa = cuda_lib
    q, k, v, w, table, pos = _case(T, hq, hkv, dim, 64, seed=hq)
    axes = pa.mrope_axes([16, 8, 8])
    for il in (False, True):
        got = pa.qk_norm_mrope(q, k, *w, table, pos, axes, 1e-6, interleaved=il)
        got += pa.qk_norm_rope(q, k, *w, table, pos[0], 1e-6, interleaved=il)
        for out, x, ww, p in zip(got, (q, k, q, k), w + w, (pos, pos, pos[:1], pos[:1])):
            ref, tol = _ref(x, ww, table, p, axes if p is pos else bytes(32), il)
            assert (np.abs(f64(out) - ref) <= tol).all()
    assert pa.device_errors() == 0
