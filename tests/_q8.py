"""Plain 64-bit implementations of the 8-bit cache and of rotation by several axes, in numpy, written
from the definitions in include/pa.h.  The tests compare the library with these."""
import numpy as np

BLOCK = 16


def decoded(codes):
    """e4m3 bytes -> fp64."""
    c = np.asarray(codes, np.int64)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e > 0, (8 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c > 127, -x, x)


_POSITIVE = decoded(np.arange(127))  # 0 .. 448, ascending


def encoded(x):
    """fp64 -> the nearest code (ties to the even one); NaN for what is not finite.  The sign of a
    zero is kept, and |x| may be at most 464, where 448 ends."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    a = np.where(finite, np.abs(x), 0)
    assert (a <= 464).all()
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    down, up = a - _POSITIVE[lo], _POSITIVE[hi] - a
    n = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(finite, n + 128 * np.signbit(x), 127).astype(np.uint8)


def scale_byte(top):
    """The smallest byte (1 at least) with top <= 448 * 2^(b - 127), by trying."""
    b = 1
    while top > 448 * 2.0 ** (b - 127):
        b += 1
    return b


def empty_cache(pages, bs, hkv, fill=0xA5, scale=0x5A):
    return (np.full((pages, bs, hkv, 256), fill, np.uint8),
            np.full((pages, -(-bs // BLOCK), hkv), scale, np.uint8))


def write(codes, scales, slots, x):
    """In place, block by block; x fp64 [T, heads, 256]."""
    pages, bs, hkv, _ = codes.shape
    blocks = {}
    for t, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < pages * bs:
            blocks.setdefault((s // bs, s % bs // BLOCK), {})[s % bs % BLOCK] = t  # the last one counts
    for (page, i), rows in blocks.items():
        at = sorted(rows)
        first, count = i * BLOCK, min(BLOCK, bs - i * BLOCK)
        for h in range(hkv):
            v = x[[rows[r] for r in at], h]
            ok = np.abs(v[np.isfinite(v)])
            need, old = scale_byte(ok.max() if ok.size else 0.0), int(scales[page, i, h])
            anew = 0 in rows or old == 255
            b = need if anew else max(old, need)
            part = codes[page, first:first + count, h]
            if not anew and b > old:
                rest = [r for r in range(count) if r not in rows]
                was = part[rest]
                part[rest] = encoded(decoded(was) * 2.0 ** (old - b))
            part[at] = encoded(v * 2.0 ** (127 - b))
            scales[page, i, h] = b


def values(codes, scales, page, offset, head):
    """pages and offsets [N] -> fp64 [N, 256]."""
    b = scales[page, offset // BLOCK, head].astype(np.float64)
    return decoded(codes[page, offset, head]) * np.where(b == 255, np.nan, 2.0 ** (b - 127))[:, None]


def keys(cache, table_row, count, head):
    codes, scales = cache
    t = np.arange(count)
    bs = codes.shape[1]
    return values(codes, scales, np.asarray(table_row)[t // bs].astype(np.int64), t % bs, head)


def attend(q, k, v, scale, visible, weight=2.0 ** -11):
    """q [M, 256], k, v [N, 256]; row i sees keys 0 .. visible[i] - 1 (one at least).  Returns the
    fp64 outputs and, per element, the bound on what the kernel may be off by:

    * the output's rounding to BF16: half a step, 2^-8 of it;
    * a weight's rounding to FP16: 2^-11 of it (and 2^-31 of the row's largest where FP16 is
      subnormal; N of those);
    * scores: products of 11 and 4 bits are exact in fp32; their sums are made in 16 steps, each off
      by 2^-22 of what is summed up at most, so 2^-18 of sum |q| |k|; exponent and exponential:
      2^-22 |x| and 2^-21.  A weight changes by that, relative, and the weights' sum by its mean;
    * the sums over tokens: 16 tokens a step, 2^-22 of what is summed up each."""
    N = k.shape[0]
    x = q @ k.T * scale
    wide = np.abs(q) @ np.abs(k).T * abs(scale)
    x[np.arange(N) >= np.asarray(visible)[:, None]] = -np.inf
    p = np.exp(x - x.max(-1, keepdims=True))
    top = p.max(-1, keepdims=True) / p.sum(-1, keepdims=True)
    p /= p.sum(-1, keepdims=True)
    out = p @ v
    d = np.where(p > 0, 1.5 * wide * 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(p > 0, x, 0)) + 2.0 ** -21, 0)
    mean = (p * d).sum(-1, keepdims=True)
    size = p @ np.abs(v)
    bound = 2.0 ** -8 * np.abs(out) + (weight + (N / 16 + 16) * 2.0 ** -22) * size
    bound += np.expm1(1.0) * ((p * d) @ np.abs(v) + mean * size)  # e^d - 1 <= (e - 1) d
    return out, 1.01 * bound + 2.0 ** -31 * top * np.abs(v).sum(0) + 1e-30


def decode(q, kc, vc, table, lens, scale):
    S, hq, _ = q.shape
    hkv = kc[0].shape[2]
    out, tol = np.zeros(q.shape), np.full(q.shape, 1e-30)
    for s in range(S):
        for g in range(hkv if lens[s] else 0):
            k, v = (keys(c, table[s], lens[s], g) for c in (kc, vc))
            h = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            out[s, h], tol[s, h] = attend(q[s, h], k, v, scale, np.full(hq // hkv, lens[s]))
    return out, tol


def prefill(q, kc, vc, table, cu, lens, causal, scale):
    hkv = kc[0].shape[2]
    G = q.shape[1] // hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        if r1 == r0:
            continue
        seen = n - (r1 - r0) + 1 + np.arange(r1 - r0) if causal else np.full(r1 - r0, n)
        for g in range(hkv):
            k, v = (keys(c, table[b], n, g) for c in (kc, vc))
            for h in range(g * G, (g + 1) * G):
                out[r0:r1, h], tol[r0:r1, h] = attend(q[r0:r1, h], k, v, scale, seen)
    return out, tol


def mrope(x, w, bias, eps, cos_sin, positions, axes, interleaved):
    """[T, H, D] fp64; positions [axes, T]."""
    T, _, dim = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + bias)
    half = cos_sin.shape[1] // 2
    out = y.copy()
    for t in range(T):
        if (positions[:, t] < 0).any():
            continue
        for i in range(half):
            row = cos_sin[positions[axes[i], t]]
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, a] = y[t, :, a] * row[i] - y[t, :, b] * row[half + i]
            out[t, :, b] = y[t, :, b] * row[i] + y[t, :, a] * row[half + i]
    return out
