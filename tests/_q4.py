"""Plain 64-bit implementations of the 4-bit cache and the steps around it, in numpy, written
from the definitions in include/pa.h.  The tests compare the library with these."""
import numpy as np
import torch

D, GROUPS, ROW = 256, 4, 144


def bf16(x):
    """fp64 -> the nearest BF16 values (ties to even), as fp64 (for finite x).  The spacing is
    2^-8 of the binade's upper end, and 2^-133 among the subnormals."""
    x = np.asarray(x, np.float64)
    q = np.maximum(np.frexp(x)[1], -125) - 8
    return np.ldexp(np.rint(np.ldexp(x, -q)), q)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def quantise(x):
    """[..., 256] -> codes [..., 256], steps and minima [..., 4]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], GROUPS, 64)
    lo, hi = g.min(-1), g.max(-1)
    s = bf16(((hi - lo).astype(np.float32) / np.float32(15)).astype(np.float64))
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.rint((g - lo[..., None]) / s[..., None])
    n = np.where(s[..., None] > 0, np.clip(n, 0, 15), 0).astype(np.int64)
    return n.reshape(x.shape), s, lo


def value(n, s, lo):
    g = n.reshape(*n.shape[:-1], GROUPS, 64)
    return (lo[..., None] + s[..., None] * g).reshape(n.shape)


def _bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def empty_cache(pages, bs, hkv, fill=0xFF):
    return np.full((pages, hkv, bs * ROW), fill, np.uint8)


def store(cache, bs, slot, head, n, s, lo):
    """One token's row of one head, byte by byte."""
    run, o = cache[slot // bs, head], slot % bs
    for d in range(D):
        g, u, j = d // 64, d % 64 // 8, d % 8
        at = o * 128 + (u ^ (o % 8)) * 16 + 4 * g + j // 2
        keep = 0x0F if j % 2 else 0xF0
        run[at] = (run[at] & keep) | (int(n[d]) << (4 * (j % 2)))
    for g in range(GROUPS):
        at = bs * 128 + o * 16 + 4 * g
        run[at:at + 2] = np.frombuffer(_bf16_bits(s[g]).tobytes(), np.uint8)
        run[at + 2:at + 4] = np.frombuffer(_bf16_bits(lo[g]).tobytes(), np.uint8)


def load(cache, bs, page, offset, head):
    """Vectorised read: pages and offsets [N] -> fp64 [N, 256], and the steps [N, 4]."""
    run = cache[page, head]
    d = np.arange(D)
    g, u, j = d // 64, d % 64 // 8, d % 8
    at = offset[:, None] * 128 + (u ^ (offset[:, None] % 8)) * 16 + 4 * g + j // 2
    raw = np.take_along_axis(run, at, 1).astype(np.int64)
    n = np.where(j % 2, raw >> 4, raw & 15)
    pairs = bs * 128 + offset[:, None] * 16 + np.arange(16)
    b = np.take_along_axis(run, pairs, 1).astype(np.uint32)
    w = ((b[:, 0::2] | (b[:, 1::2] << 8)) << 16).view(np.float32).astype(np.float64)
    return value(n, w[:, 0::2], w[:, 1::2]), w[:, 0::2]


def keys(cache, bs, table_row, count, head):
    t = np.arange(count)
    return load(cache, bs, np.asarray(table_row)[t // bs].astype(np.int64), t % bs, head)


def attend(q, k, v, scale, visible):
    """q [M, 256], k, v [N, 256]; row i sees keys 0 .. visible[i] - 1."""
    x = q @ k.T * scale
    x[np.arange(k.shape[0]) >= np.asarray(visible)[:, None]] = -np.inf
    p = np.exp(x - x.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True) @ v


def decode(q, kc, vc, bs, table, lens, scale):
    """fp64 outputs, and per element the bound on what the kernel may be off by.

    The bound: the output's rounding to BF16 (half a step, 2^-8 of it); FP16 weights (2^-11
    each, times codes of at most 15 steps; and of those below FP16's normal range, at 2^-21 of
    the largest, nothing that counts); scores in fp32 -- 64 products a group, 4 groups: at most
    2^-17 of sum |q| (|lo| + 64 s) -- which move a weight by twice their error; the exponential's
    approximation (2^-21); the sums of both (2^-17 of the largest value)."""
    S, hq, _ = q.shape
    G = hq // kc.shape[1]
    out, tol = np.zeros(q.shape), np.full(q.shape, 1e-30)
    for s in range(S):
        if lens[s] == 0:
            continue
        for h in range(hq):
            k, ks = keys(kc, bs, table[s], lens[s], h // G)
            v, vs = keys(vc, bs, table[s], lens[s], h // G)
            o = attend(q[s, h][None], k, v, scale, [lens[s]])[0]
            big = np.abs(q[s, h]).sum() * (np.abs(k).max() + 64 * ks.max()) * abs(scale)
            vmax = np.repeat(np.abs(v).reshape(-1, GROUPS, 64).max((0, 2)), 64)
            step = np.repeat(vs.max(0), 64)
            out[s, h] = o
            tol[s, h] = (2.0 ** -8 * np.abs(o) + 2.0 ** -11 * 15 * step
                         + (2 * 2.0 ** -17 * big + 2.0 ** -17 + 2.0 ** -21) * vmax) * 1.01
    return out, tol


def prefill(q, kc, vc, bs, table, cu, lens, causal, scale):
    """fp64 outputs of stacked chunks, and per element the bound on what the kernel may be off
    by: the output's rounding to BF16 (half a step, 2^-8 of it); K in FP16 (2^-11 of each value),
    which moves a row's scores by at most 2^-11 max sum |q| |k|, and fp32 sums (2^-17 of that
    sum), a weight by e^(twice that) - 1; weights and V in FP16 (2^-11 each of a value)."""
    hkv = kc.shape[1]
    G = q.shape[1] // hkv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        if r1 == r0:
            continue
        seen = n - (r1 - r0) + 1 + np.arange(r1 - r0) if causal else np.full(r1 - r0, n)
        for h in range(q.shape[1]):
            if h % G == 0:
                k, v = (keys(x, bs, table[b], n, h // G)[0] for x in (kc, vc))
            x = q[r0:r1, h]
            o = attend(x, k, v, scale, seen)
            moved = (np.abs(x) @ np.abs(k).T).max(-1, keepdims=True) * abs(scale) * (2.0 ** -11 + 2.0 ** -17)
            out[r0:r1, h] = o
            tol[r0:r1, h] = 2.0 ** -8 * np.abs(o) + (np.expm1(2 * moved) + 2.0 ** -10) * np.abs(v).max(0)
    return out, tol * 1.01 + 1e-30


def rope(x, w, bias, eps, cos_sin, positions, interleaved):
    """[T, H, D] fp64."""
    T, _, dim = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + bias)
    rot = cos_sin.shape[1]
    half = rot // 2
    out = y.copy()
    for t in range(T):
        if positions[t] < 0:
            continue
        c, s = cos_sin[positions[t], :half], cos_sin[positions[t], half:]
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, a] = y[t, :, a] * c[i] - y[t, :, b] * s[i]
            out[t, :, b] = y[t, :, b] * c[i] + y[t, :, a] * s[i]
    return out


def cos_sin_table(rows, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(rows)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def batch_prep(computed, new, tables, sizes, free, T):
    """One sequence and one token at a time; returns the outputs and whether pages ran out."""
    tables = [t.copy() for t in tables]
    lens, starts = [], [0]
    pos, own = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    slots = [np.full(T, -1, np.int64) for _ in sizes]
    taken, short = [0] * len(sizes), False
    for s, (c, n) in enumerate(zip(computed.tolist(), new.tolist())):
        n = max(n, 0)
        lens.append(c + n if n else 0)
        starts.append(starts[-1] + n)
        for g, bs in enumerate(sizes):
            mb = tables[g].shape[1]
            for blk in range(-(-c // bs), -(-(c + n) // bs) if n else 0):
                if blk >= mb:
                    break
                page = -1
                if taken[g] < len(free[g]):
                    page = free[g][taken[g]]
                    taken[g] += 1
                else:
                    short = True
                if starts[-2] + max(blk * bs - c, 0) < T:
                    tables[g][s, blk] = page
        for i in range(n):
            t = starts[-2] + i
            if t >= T:
                break
            pos[t], own[t] = c + i, s
            for g, bs in enumerate(sizes):
                blk = (c + i) // bs
                if blk < tables[g].shape[1] and tables[g][s, blk] >= 0:
                    slots[g][t] = int(tables[g][s, blk]) * bs + (c + i) % bs
    return dict(seq_lens=np.array(lens, np.int32), query_start_loc=np.array(starts, np.int32),
                positions=pos, seq_idx=own, slot_mappings=slots, tables=tables,
                pages_taken=np.array(taken, np.int32)), short
