"""What decode over the 4-bit cache may be off by, as a norm for each head and group of 64 dims,
beside the output's own rounding.  Much closer than a bound per element that charges the worst key
with the largest value: a tile that is left out, or a group whose weights lose their bits, is far
outside of it."""
import numpy as np

import _q4


def parts(cache, bs, table_row, count, head):
    """Codes [N, 256], steps and minima [N, 4] of a sequence's tokens, fp64."""
    v, s = _q4.keys(cache, bs, table_row, count, head)
    t = np.arange(count)
    run = cache[np.asarray(table_row)[t // bs].astype(np.int64), head]
    at = (bs * 128 + (t % bs)[:, None] * 16 + np.arange(16))
    b = np.take_along_axis(run, at, 1).astype(np.uint32)
    lo = ((b[:, 0::2] | (b[:, 1::2] << 8)) << 16).view(np.float32).astype(np.float64)[:, 1::2]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = (v.reshape(-1, 4, 64) - lo[..., None]) / s[..., None]
    return np.where(s[..., None] > 0, np.rint(n), 0).reshape(count, 256), s, lo


def _norms(x):  # of each group of 64
    return np.linalg.norm(x.reshape(*x.shape[:-1], 4, 64), axis=-1)


def attend(q, k, v, scale):
    """One head: q [256]; k, v (codes, steps, minima).  Returns the fp64 output [256] and, per
    group, the bound on the norm of what the kernel's result may be off by before its rounding.

    * A weight times a step is rounded to FP16: 2^-11 of it at most, and 2^-25 below the normal
      range, the largest of the group being 2^-1 at least (2^-24 of the largest).  Errors of
      different tokens are independent: four times the root of their squares, spread evenly over
      half a step (4 / sqrt(3) also covers up to five tokens that err in one direction).
    * Scores: products are exact in fp32, sums of 16 of them are added up in 4 steps a group and 6
      more, each off by 2^-23 of what it adds up, so 2^-19 of sum |q| (|lo| + s n); the
      exponential's argument and result, 2^-21 together.  The weights' sum errs the same way.
    * Sums over tokens: 2^-23 a step of 16, a warp of four taking every fourth pair of tiles."""
    (kn, ks, kl), (vn, vs, vl) = k, v
    kk, vv = _q4.value(kn, ks, kl), _q4.value(vn, vs, vl)
    x = kk @ q * scale
    p = np.exp(x - x.max())
    p /= p.sum()
    out = p @ vv
    wide = np.abs(kl).repeat(64, -1) + ks.repeat(64, -1) * kn
    e = 2.0 ** -19 * abs(scale) * (wide @ np.abs(q)) + 2.0 ** -21 + 2.0 ** -23 * np.abs(x)
    w = p[:, None] * vs
    codes = _norms(vn)
    rounding = 4 / 3 ** 0.5 * np.sqrt(((2.0 ** -11 * w * codes) ** 2).sum(0))
    rounding += 2.0 ** -24 * w.max(0) * np.sqrt((codes ** 2).sum(0)) * 4
    size = w * codes + p[:, None] * np.abs(vl) * 8
    moved = 2 * (p * e) @ (_norms(vv) + _norms(out)) + 2.0 ** -23 * (len(x) / 64 + 8) * size.sum(0)
    return out, rounding + moved


def decode(q, kc, vc, bs, table, lens, scale):
    """fp64 outputs [S, Hq, 256] and the bounds [S, Hq, 4] of decode over the caches."""
    S, hq, _ = q.shape
    hkv = kc.shape[1]
    out, bound = np.zeros(q.shape), np.zeros((S, hq, 4))
    for s in range(S):
        for g in range(hkv if lens[s] else 0):
            k, v = (parts(c, bs, table[s], lens[s], g) for c in (kc, vc))
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                out[s, h], bound[s, h] = attend(q[s, h], k, v, scale)
    return out, bound


def excess(got, ref):
    """By how much got is further from ref than its own rounding to BF16 explains: half a step
    of the larger one's binade."""
    top = np.maximum(np.abs(got), np.abs(ref))
    half = np.ldexp(1.0, np.maximum(np.frexp(top)[1], -125) - 9)
    return np.maximum(np.abs(got - ref) - half, 0)


def check(got, ref, bound):
    over = _norms(excess(got, ref))
    assert np.isfinite(got).all()
    with np.errstate(divide="ignore", invalid="ignore"):
        worst = np.nanmax(np.where(over > 0, over / bound, 0), initial=0)
    assert (over <= bound).all(), worst
    return worst
