"""The 8-bit cache where its kernels change their ways: writes past the longest range of a CTA and in
pools past what the block map tells apart, the two forms of the decode on one batch, and V far below
its head's largest."""
import numpy as np
import pytest
import torch

import _q8
from _q4 import f64
from test_gpu_q8 import _case, _check_decode, _decode, _down, _plain_caches, _refill, _rows

pytestmark = pytest.mark.gpu


def _random_caches(pa, pages, bs, hkv, seed):
    """Caches of any codes (NaN among them) under scales of 100 to 139: K, V, their scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes, scales = pa.q8_cache_shapes(pages, bs, hkv)
    return [torch.randint(0, 256, codes, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
            for _ in range(2)] + [torch.randint(100, 140, scales, generator=g, device="cuda", dtype=torch.uint8)
                                  for _ in range(2)]


def _bytes(cache):
    return [c.view(torch.uint8) for c in cache]


# A CTA takes at most 256 tokens, which the grid's two CTAs an SM exceed from 39000 (8 heads) to 78000
# tokens on.  Straight calls of a few thousand tokens, which the other tests hold to the plain form, give
# the bits that the one call has to give.
@pytest.mark.parametrize("T,hkv,bs", [(80001, 1, 16), (90000, 3, 100), (41000, 9, 64)])
@pytest.mark.parametrize("order", ["straight", "shuffled"])
def test_write_past_the_longest_range(cuda_lib, T, hkv, bs, order):
    pa = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = -(-T // bs) + 2
    key, val = (torch.randn(T, hkv, 256, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    key[::7] *= 100
    slots = torch.randperm(pages, generator=g, device="cuda")[torch.arange(T, device="cuda") // bs] * bs \
        + torch.arange(T, device="cuda") % bs
    want, got = (_random_caches(pa, pages, bs, hkv, 1) for _ in range(2))
    step = 4000 // bs * bs  # (whole pages, so that a block's tokens come in one call)
    for t in range(0, T, step):
        pa.reshape_and_cache_q8(key[t:t + step], val[t:t + step], *want, slots[t:t + step])
    if order == "shuffled":
        p = torch.randperm(T, generator=g, device="cuda")
        key, val, slots = key[p], val[p], slots[p]
    # Tokens of which a later one has the slot: the first's, in the last token's block or far from it.
    key, val = torch.cat([key[-3:], key]), torch.cat([val[-3:] * 1000, val])
    slots = torch.cat([slots[[-1, T // 2, 0]], slots])
    pa.reshape_and_cache_q8(key, val, *got, slots)
    for a, b in zip(_bytes(got), _bytes(want)):
        assert torch.equal(a, b)
    assert pa.device_errors() == 0


# Slots that are 262144 apart share a bit of the CTAs' block maps.
@pytest.mark.parametrize("bs,pages", [(16, 50000), (832, 1000), (7, 90000)])
@pytest.mark.parametrize("T", [40, 1500, 6000])
def test_write_in_a_large_pool(cuda_lib, bs, pages, T):
    pa = cuda_lib
    rng = np.random.default_rng(T + bs)
    wrap = 16384 * 16
    low = rng.choice(wrap // 2, T // 2, replace=False)
    slots = np.concatenate([low, low + wrap])
    slots[1::9] += wrap if bs != 7 else 0  # (three on a bit; each slot once, or its last token counts)
    slots = rng.permutation(slots)
    assert slots.max() < pages * bs
    key, val = _rows(len(slots), 1, 3), _rows(len(slots), 1, 4, "outliers")
    cache = _random_caches(pa, pages, bs, 1, 2)
    want = [c.clone() for c in _bytes(cache)]
    used = np.unique(slots // bs)  # the plain form on these pages alone
    at = torch.from_numpy(used).cuda()
    near = np.searchsorted(used, slots // bs) * bs + slots % bs
    for x, i in ((key, 0), (val, 1)):
        codes, scales = want[i][at].cpu().numpy(), want[2 + i][at].cpu().numpy()
        _q8.write(codes, scales, near, f64(x))
        want[i][at], want[2 + i][at] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    pa.reshape_and_cache_q8(key.cuda(), val.cuda(), *cache, torch.from_numpy(slots).cuda())
    for a, b in zip(_bytes(cache), want):
        assert torch.equal(a, b)
    assert pa.device_errors() == 0


# The bound on the lengths picks the decode's form: a cluster a pair, or the cut row and the merge.
@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (832, 24, 4, [1 + (i * 67) % 300 for i in range(16)]), (64, 24, 4, [1000, 999, 3, 0]),
    (16, 8, 2, [(i * 131) % 700 for i in range(16)]), (48, 6, 1, [1, 300]), (7, 16, 8, [0, 77, 8, 0, 130]),
])
def test_decode_under_a_tight_and_a_loose_bound(cuda_lib, bs, hq, hkv, lens):
    pa = cuda_lib
    c = _case(pa, lens, bs, hq, hkv, seed=len(lens), max_blocks=-(-40000 // bs))
    tight = _decode(pa, c)
    loose = _decode(pa, c, max_len=40000)
    _check_decode(tight, c)
    _check_decode(loose, c)
    # Both are the fp32 attention over FP16 weights, rounded to BF16 once.
    assert (tight.float() - loose.float()).abs().max() <= 2.0 ** -7 * tight.float().abs().max()
    assert pa.device_errors() == 0


# V's codes become FP16 in steps of 2^-24 at least, times 2^(6 - 127) and the head's largest scale: off
# by half such a step, 2^-31 of 2^(b - 127), where a block lies more than 2^15 below.  The rows that do not
# see the large block are held to that alone; from 2^21 on its codes pass FP16's smallest normal value.
@pytest.mark.parametrize("apart", [16, 20, 24, 28, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_of_blocks_far_below_the_largest(cuda_lib, apart, causal):
    pa = cuda_lib
    c = _case(pa, [64], 16, 2, 2, seed=apart, rows=32)
    rng = np.random.default_rng(apart)
    v = rng.standard_normal((64, 2, 256))
    v[48:, 0] *= 2.0 ** apart
    _refill(pa, c, rng.standard_normal((64, 2, 256)), v)
    out = f64(pa.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], 32, causal, 0.0625))
    ref, tol = _q8.prefill(f64(c["q"]), *_plain_caches(c), c["table"], [0, 32], [64], causal, 0.0625)
    _, scales = _down(*c["cache"][1::2])
    top = scales[c["table"][0]].astype(np.float64).max((0, 1))  # of each head
    tol += 2.0 ** -31 * 2.0 ** (top[:, None] - 127)
    assert (np.abs(out - ref) <= tol).all()
    if causal:
        # Rows 0 .. 15 see keys before 48 alone, so none of the large block's values is in their bound.
        ref, tol = _q8.prefill(f64(c["q"][:16]), *_plain_caches(c), c["table"], [0, 16], [48], True, 0.0625)
        tol += 2.0 ** -31 * 2.0 ** (top[:, None] - 127)
        assert (np.abs(out[:16] - ref) <= tol).all()
        assert (tol < np.abs(ref)).mean() > 0.5  # (zeros would not pass)
