"""Decode over the 4-bit cache against 64 bits under a bound on each head's and group's error norm
(_q4_bounds): ordinary data, values of V of very uneven size, and scores that are all alike, where
every token counts the same and one left out or counted twice shows."""
import numpy as np
import pytest
import torch

import _q4
import _q4_bounds
from test_gpu_q4 import _case, _decode

pytestmark = pytest.mark.gpu


def _check(out, c, scale=0.0625):
    ref, bound = _q4_bounds.decode(_q4.f64(c["q"]), c["kc"].cpu().numpy(), c["vc"].cpu().numpy(), c["bs"],
                                   c["table"], c["lens"].cpu().numpy(), scale)
    return _q4_bounds.check(_q4.f64(out), ref, bound)


def _bf(x):
    return x.to(torch.bfloat16).contiguous()


@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (832, 24, 4, [1701]),
    (784, 6, 1, [783, 785, 1568]),
    (16, 32, 8, [1, 2, 15, 16, 17, 0, 31, 33, 200]),
    (7, 5, 1, [1, 6, 7, 8, 99]),
    (100, 14, 2, [99, 100, 101, 350]),
    (16, 16, 8, [(i * 389) % 601 for i in range(33)] + [0, 0, 1, 1, 2, 0, 599, 0]),
    (64, 16, 4, [0, 20001, 0]),
])
def test_decode_within_the_norm_bound(cuda_lib, bs, hq, hkv, lens):
    c = _case(cuda_lib, lens, bs, hq, hkv, seed=3 * len(lens) + bs)
    _check(_decode(cuda_lib, c), c)
    assert cuda_lib.device_errors() == 0


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_decode_scales_within_the_norm_bound(cuda_lib, scale):
    c = _case(cuda_lib, [300, 17], 64, 6, 1, seed=9)
    _check(_decode(cuda_lib, c, scale), c, scale)


@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (832, 24, 4, [1701]), (16, 6, 1, [5000]), (784, 8, 8, [785, 0, 1, 2999]), (7, 5, 1, [333, 6]),
    (16, 8, 8, [(i * 577) % 1201 for i in range(34)]), (48, 16, 4, [20001, 17]),
])
def test_decode_flat_scores_count_every_token(cuda_lib, bs, hq, hkv, lens):
    # Token t has one value, 15 in dim t % 256 (a step of 1, exact): dim d of the mean counts the
    # tokens of that dim, so that one token more or less moves it by 256 / length of it at least.
    pa = cuda_lib
    c = _case(pa, lens, bs, hq, hkv, seed=bs)
    c["q"].zero_()
    v = torch.zeros(sum(lens), hkv, 256, device="cuda")
    t = torch.cat([torch.arange(n) for n in lens]).cuda()
    v[torch.arange(sum(lens), device="cuda"), :, t % 256] = 15
    k = torch.randn(sum(lens), hkv, 256, device="cuda")
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    out = _q4.f64(_decode(pa, c))
    for s, n in enumerate(lens):
        want = 15.0 * np.bincount(np.arange(n) % 256, minlength=256) / max(n, 1)
        # a rounding to BF16 (2^-8), and to FP16 the same weight for all (2^-11)
        assert (np.abs(out[s] - want) <= want * (2.0 ** -8 + 2.0 ** -10)).all(), (s, n)


@pytest.mark.parametrize("apart", [2.0 ** 20, 2.0 ** 24, 2.0 ** 28, 2.0 ** 60])
@pytest.mark.parametrize("lens", [[500], [9000, 40]])
def test_decode_uneven_groups(cuda_lib, apart, lens):
    # Groups of V whose sizes are far apart: each keeps the precision of its own.
    pa = cuda_lib
    c = _case(pa, lens, 64, 6, 1, seed=11)
    N = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(N, 1, 4, 64, generator=g, device="cuda")
    v *= torch.tensor([apart, 1.0, 1 / apart, apart ** 0.5], device="cuda")[:, None]
    k = torch.randn(N, 1, 256, generator=g, device="cuda")
    pa.reshape_and_cache_q4(_bf(k), _bf(v.flatten(-2)), c["kc"], c["vc"], c["slots"])
    _check(_decode(pa, c), c)


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 24, 2.0 ** 28, 2.0 ** 60])
@pytest.mark.parametrize("at", [0, 250, 499])
def test_decode_large_token_of_negligible_weight(cuda_lib, size, at):
    # One token whose V is far larger than the others' and whose weight is e^-60 or so.
    pa = cuda_lib
    c = _case(pa, [500], 64, 4, 1, seed=12)
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(256, generator=g, device="cuda")
    c["q"] = _bf(u + 0.05 * torch.randn(1, 4, 256, generator=g, device="cuda"))
    k = torch.randn(500, 1, 256, generator=g, device="cuda")
    v = torch.randn(500, 1, 256, generator=g, device="cuda")
    k[at] = -u * (60 / 0.0625 / float(u @ u))
    v[at] *= size
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    _check(_decode(pa, c), c)


@pytest.mark.parametrize("small,large", [(1e-24, 1e15), (1e-30, 1e30)])
def test_decode_tiny_steps_beside_a_large_constant_group(cuda_lib, small, large):
    pa = cuda_lib
    c = _case(pa, [300], 64, 6, 1, seed=13)
    g = torch.Generator(device="cuda").manual_seed(3)
    v = torch.randn(300, 1, 256, generator=g, device="cuda") * small
    v[:, :, 64:128] = torch.randn(300, 1, 1, generator=g, device="cuda") * large
    k = torch.randn(300, 1, 256, generator=g, device="cuda")
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    _check(_decode(pa, c), c)


@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e30, 3e36])
def test_decode_sizes_of_v(cuda_lib, size):
    c = _case(cuda_lib, [700, 3], 64, 6, 1, seed=14, scale_v=size)
    _check(_decode(cuda_lib, c), c)


def test_decode_scores_that_grow_along_the_keys(cuda_lib):
    # The largest score moves again and again, and with it the sums of every group.
    pa = cuda_lib
    n = 3000
    c = _case(pa, [n], 64, 6, 1, seed=15)
    g = torch.Generator(device="cuda").manual_seed(4)
    grow = torch.linspace(0, 24, n, device="cuda")[:, None, None]
    k = torch.randn(n, 1, 256, generator=g, device="cuda") * (1 + grow)
    v = torch.randn(n, 1, 256, generator=g, device="cuda") * torch.exp2(2 * grow)
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    for scale in (0.0625, 0.01, -0.03):
        _check(_decode(pa, c, scale), c, scale)


# ------------------------------------------------------------------------------ prefill
def _prefill_uneven(pa, rows, n, v, seed=0, scale=0.0625, far=None):
    """A causal chunk over values v [n, 2, 256]; returns its outputs and the plain ones."""
    c = _case(pa, [n], 64, 12, 2, seed=seed, rows=rows)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(n, 2, 256, generator=g, device="cuda")
    if far is not None:  # a key that outweighs no other: scores 60 below in every row
        u = torch.randn(256, generator=g, device="cuda")
        c["q"] = _bf(u + 0.05 * torch.randn(rows, 12, 256, generator=g, device="cuda"))
        k[far] = -u * (60 / 0.0625 / float(u @ u))
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    out = pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], n - rows, True, scale)
    ref, tol = _q4.prefill(_q4.f64(c["q"]), c["kc"].cpu().numpy(), c["vc"].cpu().numpy(), 64, c["table"],
                           [0, rows], [n], True, scale)
    assert pa.device_errors() == 0
    return _q4.f64(out), ref, tol


def _group_errors(out, ref):
    """Error norm over reference norm of each group of 64 dims, all rows and heads together."""
    norm = lambda x: np.linalg.norm(x.reshape(-1, 4, 64), axis=(0, 2))
    return norm(out - ref) / norm(ref)


# The whole of a group's errors: a rounding to BF16, at most 2^-8 / sqrt(3) where errors are spread
# evenly over half a step, and a fifth for the FP16 operands (2^-11 / sqrt(3) each).
GROUP = 2.0 ** -8 / 3 ** 0.5 * 1.2


@pytest.mark.parametrize("apart", [2.0 ** 8, 2.0 ** 16, 2.0 ** 22])
def test_prefill_uneven_groups(cuda_lib, apart):
    # Down to 2^-28 of the head's largest value FP16 keeps its 11 bits.
    g = torch.Generator(device="cuda").manual_seed(5)
    v = torch.randn(700, 2, 4, 64, generator=g, device="cuda")
    v *= torch.tensor([apart, 1.0, 4.0, apart ** 0.5], device="cuda")[:, None]
    out, ref, tol = _prefill_uneven(cuda_lib, 200, 700, v.flatten(-2), seed=21)
    assert (np.abs(out - ref) <= tol).all()
    assert (_group_errors(out, ref) <= GROUP).all(), _group_errors(out, ref)


@pytest.mark.parametrize("at", [0, 300, 499])
def test_prefill_large_token_of_negligible_weight(cuda_lib, at):
    g = torch.Generator(device="cuda").manual_seed(6)
    v = torch.randn(700, 2, 256, generator=g, device="cuda")
    v[at] *= 2.0 ** 20
    out, ref, _ = _prefill_uneven(cuda_lib, 200, 700, v, seed=22, far=at)
    assert (_group_errors(out, ref) <= GROUP).all(), _group_errors(out, ref)


def test_prefill_values_below_the_range_of_their_head(cuda_lib):
    # A group 2^-36 times as large as another: off by up to 2^-39 of the head's largest value, and
    # the others keep their own.
    g = torch.Generator(device="cuda").manual_seed(7)
    v = torch.randn(700, 2, 4, 64, generator=g, device="cuda")
    v *= torch.tensor([1.0, 2.0 ** -36, 0.5, 2.0 ** -10], device="cuda")[:, None]
    out, ref, tol = _prefill_uneven(cuda_lib, 200, 700, v.flatten(-2), seed=23)
    largest = float(v.abs().max()) * 1.1  # (and what the quantiser adds)
    assert (np.abs(out - ref) <= tol + 2.0 ** -39 * largest).all()
    assert (_group_errors(out, ref)[[0, 2, 3]] <= GROUP).all(), _group_errors(out, ref)


# ------------------------------------------------------------------------------ one token alone
@pytest.mark.parametrize("scale_v", [1e-30, 1.0, 1e30])
def test_decode_of_one_token_is_its_row(cuda_lib, scale_v):
    # Its weight p is a power of two but for the rounding of the exponent's argument (m + 8, so 2^-21
    # where m is below 8), and p s in FP16 is exact: before its rounding the result is off by 2^-20
    # of |lo| + s n at most.
    pa = cuda_lib
    c = _case(pa, [1] * 40, 16, 16, 4, seed=24, scale_v=scale_v)
    out, cache = _q4.f64(_decode(pa, c)), c["vc"].cpu().numpy()
    for s in range(40):
        for g in range(4):
            n, step, lo = (x[0] for x in _q4_bounds.parts(cache, 16, c["table"][s], 1, g))
            want = _q4.value(n[None], step[None], lo[None])
            size = np.abs(lo).repeat(64) + step.repeat(64) * n
            assert (_q4_bounds.excess(out[s, 4 * g:4 * g + 4], want) <= 2.0 ** -20 * size).all(), (s, g)


@pytest.mark.parametrize("n,at", [(3000, 0), (3000, 1777), (3000, 2999), (40, 20), (9000, 8190)])
def test_decode_of_a_token_that_outweighs_the_others_is_its_row(cuda_lib, n, at):
    pa = cuda_lib
    c = _case(pa, [n], 64, 8, 2, seed=25)
    g = torch.Generator(device="cuda").manual_seed(8)
    u = torch.randn(256, generator=g, device="cuda")
    c["q"] = _bf(u.expand(1, 8, 256))
    k, v = (torch.randn(n, 2, 256, generator=g, device="cuda") for _ in range(2))
    k[at] += u * (200 / 0.0625 / float(u @ u))  # e^200: the others' weights are 0 in fp32
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    row = pa.gather_cache_q4(c["kc"], c["vc"], c["slots"][at:at + 1])[1]
    assert torch.equal(_decode(pa, c), row.repeat_interleave(4, 1))


@pytest.mark.parametrize("bs,hq,hkv,rows,lens", [
    (64, 12, 2, [300], [1500]), (832, 24, 4, [40], [9000]), (16, 16, 8, [1, 129, 0, 64, 200], [700, 129, 33, 65, 1300]),
    (7, 5, 1, [128, 17], [128, 300])])
def test_prefill_flat_scores_count_every_token(cuda_lib, bs, hq, hkv, rows, lens):
    # As the decode's: dim d of row i counts the tokens t <= its position with t % 256 == d.
    pa = cuda_lib
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    c = _case(pa, lens, bs, hq, hkv, seed=bs, rows=cu[-1])
    c["q"].zero_()
    v = torch.zeros(sum(lens), hkv, 256, device="cuda")
    t = torch.cat([torch.arange(n) for n in lens]).cuda()
    v[torch.arange(sum(lens), device="cuda"), :, t % 256] = 15
    pa.reshape_and_cache_q4(_bf(torch.randn(sum(lens), hkv, 256, device="cuda")), _bf(v), c["kc"], c["vc"], c["slots"])
    out = _q4.f64(pa.prefill_varlen_q4(c["q"], c["kc"], c["vc"], c["bt"], cu, lens, True, 0.0625))
    for b, n in enumerate(lens):
        seen = n - rows[b] + 1 + np.arange(rows[b])  # keys of each row
        count = (seen[:, None] + 255 - np.arange(256)) // 256
        want = (15.0 * count / seen[:, None])[:, None]
        got = out[cu[b]:cu[b + 1]]
        assert (np.abs(got - want) <= want * (2.0 ** -8 + 2.0 ** -10)).all(), b
    assert pa.device_errors() == 0
