"""The decode bound itself, on the CPU: it takes what the kernel's arithmetic gives and refuses a
result with a tile left out or a group whose weights were rounded away."""
import numpy as np
import pytest

import _q4
import _q4_bounds


def _parts(rng, N, scale=np.ones(4), peaks=0.0):
    x = rng.standard_normal((N, 256)) * np.repeat(scale, 64)
    x *= 1 + 7 * (rng.random((N, 1)) < peaks)
    return _q4.quantise(_q4.bf16(x))


def _fp16(x, top):
    """x as FP16 after a power of two has brought `top` to [2^-1, 1), as fp64."""
    f = 2.0 ** -np.frexp(top)[1]
    return (x * f).astype(np.float16).astype(np.float64) / f


def _result(q, k, v, scale, keep=None, own=True):
    """As the kernel rounds: weights times steps in FP16, relative to the group's largest, or to
    one largest of all groups."""
    x = _q4.value(*k) @ q * scale
    p = np.exp(x - x.max())
    w = p[:, None] * v[1]
    top = w.max(0) if own else np.broadcast_to(p.max() * v[1].max(), 4)
    w = np.stack([_fp16(w[:, g], top[g]) for g in range(4)], 1)
    t = np.ones(len(p), bool) if keep is None else keep
    o = (w[t].repeat(64, 1) * v[0][t]).sum(0) + p[t] @ v[2].repeat(64, 1)[t]
    return _q4.bf16(o / p[t].sum())


@pytest.mark.parametrize("N,peaks,scale", [(1701, 0.0, 0.0625), (333, 0.05, 0.0625), (40, 0.0, 1.0),
                                           (1, 0.0, 0.0625), (700, 0.05, -0.0625)])
def test_bound_takes_the_kernels_rounding(N, peaks, scale):
    rng = np.random.default_rng(N)
    k, v, q = _parts(rng, N, peaks=peaks), _parts(rng, N), _q4.bf16(rng.standard_normal(256))
    ref, bound = _q4_bounds.attend(q, k, v, scale)
    _q4_bounds.check(_result(q, k, v, scale)[None], ref[None], bound[None])


@pytest.mark.parametrize("N", [333, 700, 1701])
def test_bound_refuses_every_missing_tile(N):
    rng = np.random.default_rng(N)
    k, v, q = _parts(rng, N), _parts(rng, N), _q4.bf16(rng.standard_normal(256))
    ref, bound = _q4_bounds.attend(q, k, v, 0.0625)
    for t in range(0, N, 16):
        keep = np.ones(N, bool)
        keep[t:t + 16] = False
        with pytest.raises(AssertionError):
            _q4_bounds.check(_result(q, k, v, 0.0625, keep)[None], ref[None], bound[None])


@pytest.mark.parametrize("apart", [2.0 ** 24, 2.0 ** 28])
def test_bound_refuses_one_reference_for_uneven_groups(apart):
    rng = np.random.default_rng(1)
    q = _q4.bf16(rng.standard_normal(256))
    k, v = _parts(rng, 500), _parts(rng, 500, np.array([apart, 1, 4, apart / 16]))
    ref, bound = _q4_bounds.attend(q, k, v, 0.0625)
    _q4_bounds.check(_result(q, k, v, 0.0625)[None], ref[None], bound[None])
    with pytest.raises(AssertionError):
        _q4_bounds.check(_result(q, k, v, 0.0625, own=False)[None], ref[None], bound[None])
