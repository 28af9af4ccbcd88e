"""The 8-bit cache on the GPU: writes and reads bit for bit, decode and prefill against the
plain 64-bit attention over the values the cache stands for."""
import numpy as np
import pytest
import torch

import _q8
from _q4 import f64

pytestmark = pytest.mark.gpu


def _bf(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _up(cache):
    """(codes, scales) of numpy -> the tensors that the calls take."""
    return torch.from_numpy(cache[0]).cuda().view(torch.float8_e4m3fn), torch.from_numpy(cache[1]).cuda()


def _down(codes, scales):
    return codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()


def _same(codes, scales, want, msg=""):
    got = _down(codes, scales)
    assert np.array_equal(got[1], want[1]), msg + ": scales"
    assert np.array_equal(got[0], want[0]), msg + ": codes"


def _rows(T, hkv, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, 256, generator=g)
    if kind == "outliers":
        x[:, :, ::37] *= 60
        x[::5] *= 1000
    elif kind == "zeros":
        x[::2] = 0
        x[1::4] *= -0.0
    elif kind == "ties":  # halves between codes, and tops at 448 and just past it
        x = torch.randint(-63, 64, x.shape, generator=g) / 4.0
        x[0, 0, 0], x[-1, -1, 5] = 448.0, -450.0
    elif kind == "tiny":
        x *= 1e-38
    elif kind == "huge":
        x *= 8e37
    elif kind == "wide":  # forty binades
        x *= 2.0 ** torch.randint(-30, 10, x.shape, generator=g)
    elif kind == "growing":
        x *= 2.0 ** torch.arange(T)[:, None, None].clamp(max=60)
    return x.to(torch.bfloat16)


KINDS = ["normal", "outliers", "zeros", "ties", "tiny", "huge", "wide", "growing"]


# ------------------------------------------------------------------------------ writes and reads
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs,hkv,T", [(16, 4, 23), (1, 1, 3), (7, 2, 16), (40, 5, 60), (832, 4, 33)])
def test_write_matches_plain_bits(cuda_lib, kind, bs, hkv, T):
    # Slots at random, in several calls: blocks are begun, filled in any order and grow.
    pa = cuda_lib
    key, val = _rows(T, hkv, 1, kind), _rows(T, hkv, 2, kind)
    pages = -(-T // bs) + 2
    slots = torch.randperm(min(pages * bs, 2 * T + 20), generator=torch.Generator().manual_seed(3))[:T]
    want = [_q8.empty_cache(pages, bs, hkv) for _ in range(2)]
    kc, ks = _up(want[0])
    vc, vs = _up(want[1])
    cuts = [0, 1, T // 3, T // 3 + 2, T]
    for a, b in zip(cuts, cuts[1:]):
        for x, c in zip((key, val), want):
            _q8.write(*c, slots[a:b], f64(x[a:b]))
        pa.reshape_and_cache_q8(key[a:b].cuda(), val[a:b].cuda(), kc, vc, ks, vs, slots[a:b].cuda())
        _same(kc, ks, want[0], f"K {a}")
        _same(vc, vs, want[1], f"V {a}")
    ko, vo = pa.gather_cache_q8(kc, vc, ks, vs, slots.cuda())
    for got, c in ((ko, want[0]), (vo, want[1])):
        for h in range(hkv):
            v = _q8.values(*c, slots.numpy() // bs, slots.numpy() % bs, h)
            # exact but for BF16's subnormals (steps of 2^-133), and its overflow; NaN for the infinities
            # that the largest kind has among its values
            g, big, nan = f64(got[:, h]), np.abs(v) > 3.39e38, np.isnan(v)
            assert np.array_equal(np.isnan(g), nan) and np.isinf(g[big]).all()
            assert (np.abs(g - v)[~big & ~nan] <= 2.0 ** -134).all()
    assert pa.device_errors() == 0


# (Heads that do not divide among the CTAs of a range; ranges of more than a warp's tokens.)
@pytest.mark.parametrize("T,hkv,bs", [(1500, 2, 16), (2500, 1, 64), (5000, 2, 7), (700, 9, 48), (20000, 5, 16),
                                      (12000, 7, 20)])
@pytest.mark.parametrize("order", ["straight", "shuffled"])
def test_write_many_tokens_in_any_order(cuda_lib, T, hkv, bs, order):
    pa = cuda_lib
    g = torch.Generator().manual_seed(T)
    key, val = _rows(T, hkv, T), _rows(T, hkv, T + 1, "outliers")
    pages = -(-T // bs) + 3
    at = torch.randperm(pages, generator=g)[torch.arange(T) // bs] * bs + torch.arange(T) % bs
    if order == "shuffled":
        at = at[torch.randperm(T, generator=g)]
    at[T // 3] = -5
    want = [_q8.empty_cache(pages, bs, hkv, scale=120) for _ in range(2)]
    (kc, ks), (vc, vs) = _up(want[0]), _up(want[1])
    for x, c in zip((key, val), want):
        _q8.write(*c, at, f64(x))
    pa.reshape_and_cache_q8(key.cuda(), val.cuda(), kc, vc, ks, vs, at.cuda())
    _same(kc, ks, want[0], "K")
    _same(vc, vs, want[1], "V")
    assert pa.device_errors() == 0


def test_write_one_slot_twice_the_last_token_counts(cuda_lib):
    pa = cuda_lib
    T, hkv, bs = 3000, 2, 16
    key, val = _rows(T, hkv, 5), _rows(T, hkv, 6)
    key[7] *= 1e6  # ignored: its slot comes again, far behind
    slots = torch.arange(T) + 16
    slots[2900], slots[2999], slots[3], slots[40] = 23, 23, 21, 21
    want = [_q8.empty_cache(T // bs + 3, bs, hkv) for _ in range(2)]
    (kc, ks), (vc, vs) = _up(want[0]), _up(want[1])
    for x, c in zip((key, val), want):
        _q8.write(*c, slots, f64(x))
    pa.reshape_and_cache_q8(key.cuda(), val.cuda(), kc, vc, ks, vs, slots.cuda())
    _same(kc, ks, want[0])
    _same(vc, vs, want[1])


@pytest.mark.parametrize("old", [0, 1, 100, 127, 200, 254, 255])
def test_write_over_any_old_scale(cuda_lib, old):
    pa = cuda_lib
    hkv, bs = 2, 16
    g = np.random.default_rng(old)
    for first in (0, 3):
        want = [_q8.empty_cache(2, bs, hkv, scale=old) for _ in range(2)]
        for c in want:  # every code, NaN among them
            c[0][:] = g.integers(0, 256, c[0].shape, dtype=np.uint8)
        (kc, ks), (vc, vs) = _up(want[0]), _up(want[1])
        key, val = _rows(4, hkv, 8), _rows(4, hkv, 9, "huge")
        slots = torch.arange(first, first + 4)
        for x, c in zip((key, val), want):
            _q8.write(*c, slots, f64(x))
        pa.reshape_and_cache_q8(key.cuda(), val.cuda(), kc, vc, ks, vs, slots.cuda())
        _same(kc, ks, want[0])
        _same(vc, vs, want[1])


def test_write_non_finite_values_are_nan_and_leave_the_scale(cuda_lib):
    pa = cuda_lib
    x = _rows(20, 1, 5)
    bad = torch.zeros(20, 256, dtype=torch.bool)
    for t, d, v in ((0, 3, "nan"), (1, 70, "inf"), (1, 71, "-inf"), (9, 255, "nan"), (17, 0, "inf")):
        x[t, 0, d] = float(v)
        bad[t, d] = True
    x[18:] = float("nan")  # a block of nothing else behind 16, 17
    bad[18:] = True
    want = _q8.empty_cache(2, 16, 1)
    _q8.write(*want, range(20), f64(x))
    (kc, ks), (vc, vs) = _up(_q8.empty_cache(2, 16, 1)), _up(_q8.empty_cache(2, 16, 1))
    slots = torch.arange(20, device="cuda")
    pa.reshape_and_cache_q8(x.cuda(), x.cuda(), kc, vc, ks, vs, slots)
    _same(kc, ks, want)
    _same(vc, vs, want)
    for o in pa.gather_cache_q8(kc, vc, ks, vs, slots):
        assert torch.equal(torch.isnan(o[:, 0]).cpu(), bad)


def test_write_and_gather_padding_bounds_and_strides(cuda_lib):
    pa = cuda_lib
    T, hkv, bs, pages = 6, 2, 20, 3
    packed = torch.randn(T, 3 * hkv * 256, device="cuda").to(torch.bfloat16)
    key = packed[:, hkv * 256:2 * hkv * 256].unflatten(1, (hkv, 256))
    val = packed[:, 2 * hkv * 256:].unflatten(1, (hkv, 256))
    codes, scales = pa.q8_cache_shapes(pages, bs, hkv)
    both = torch.zeros(codes[:1] + (2,) + codes[1:], dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sboth = torch.zeros(scales[:1] + (2,) + scales[1:], dtype=torch.uint8, device="cuda")
    kc, vc = both.unbind(1)  # pages twice as far apart
    ks, vs = sboth.unbind(1)
    slots = torch.tensor([5, -1, 59, -7, 38, pages * bs], device="cuda")
    pa.reshape_and_cache_q8(key, val, kc, vc, ks, vs, slots)
    assert pa.device_errors() == pa.DEVERR_SLOT
    plain = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
    plain[:2] = [c.view(torch.float8_e4m3fn) for c in plain[:2]]
    ok = torch.tensor([0, 2, 4], device="cuda")
    pa.reshape_and_cache_q8(key[ok], val[ok], *plain, slots[ok])
    for a, b in zip((kc, vc, ks, vs), plain):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    ko = torch.full((T, hkv, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pa.gather_cache_q8(kc, vc, ks, vs, slots, ko, vo)
    assert pa.device_errors() == pa.DEVERR_SLOT
    assert not ko[[1, 3, 5]].any() and not vo[[1, 3, 5]].any()
    k1, v1 = pa.gather_cache_q8(*plain, slots[ok])
    assert torch.equal(ko[ok], k1) and torch.equal(vo[ok], v1)
    pa.reshape_and_cache_q8(key[:0], val[:0], *plain, slots[:0])  # no tokens
    assert pa.gather_cache_q8(*plain, slots[:0])[0].shape == (0, hkv, 256)
    far = torch.full((3000,), pages * bs + 2**40, device="cuda")
    far[2999] = 2
    assert not pa.gather_cache_q8(*plain, far)[0][:2999].any()
    assert pa.device_errors() == pa.DEVERR_SLOT


# ------------------------------------------------------------------------------ decode
def _case(pa, lens, bs, hq, hkv, seed=0, rows=None, scale_k=1.0, scale_v=1.0, spare=2, max_blocks=None):
    """Sequences in a shuffled pool whose unused places hold NaN codes under NaN scales."""
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    pool = sum(need) + spare
    perm = rng.permutation(pool)
    width = max(max(need), 1) if max_blocks is None else max_blocks
    table = np.full((len(lens), width), -1, np.int32)
    at, slots = 0, []
    for s, m in enumerate(need):
        table[s, :m] = perm[at:at + m]
        at += m
        t = np.arange(lens[s])
        slots.append(table[s, t // bs].astype(np.int64) * bs + t % bs)
    slots = torch.from_numpy(np.concatenate(slots) if slots else np.zeros(0, np.int64)).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = slots.numel()
    k = torch.randn(N, hkv, 256, generator=g, device="cuda") * scale_k
    v = torch.randn(N, hkv, 256, generator=g, device="cuda") * scale_v
    k *= 1 + 7 * (torch.rand(N, hkv, 1, generator=g, device="cuda") < 0.05)
    codes, scales = pa.q8_cache_shapes(pool, bs, hkv)
    cache = [torch.full(s, 0xFF, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
    cache[:2] = [c.view(torch.float8_e4m3fn) for c in cache[:2]]
    pa.reshape_and_cache_q8(k.to(torch.bfloat16), v.to(torch.bfloat16), *cache, slots)
    q = torch.randn(len(lens) if rows is None else rows, hq, 256, generator=g, device="cuda").to(torch.bfloat16)
    return dict(q=q, cache=cache, table=table, bt=torch.from_numpy(table).cuda(), slots=slots, bs=bs,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _plain_caches(c):
    kc, vc, ks, vs = c["cache"]
    return _down(kc, ks), _down(vc, vs)


def _decode(pa, c, scale=0.0625, max_len=None, **kw):
    return pa.decode_q8(c["q"], *c["cache"], c["bt"], c["lens"], scale,
                        max_len or max(1, int(c["lens"].max())), **kw)


def _check_decode(out, c, scale=0.0625):
    ref, tol = _q8.decode(f64(c["q"]), *_plain_caches(c), c["table"], c["lens"].cpu().numpy(), scale)
    d = np.abs(f64(out) - ref)
    assert np.isfinite(d).all()
    assert (d <= tol).all(), (d.max(), (d / tol).max())


@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (832, 24, 4, [1701]),
    (832, 24, 4, [831, 832, 833, 1]),
    (784, 6, 1, [783, 785, 1568]),
    (16, 32, 8, [1, 2, 15, 16, 17, 0, 31, 33, 200]),
    (16, 1, 1, [5000]),
    (64, 16, 2, [63, 64, 65, 0, 0, 640]),
    (7, 5, 1, [1, 6, 7, 8, 99]),
    (1, 3, 3, [1, 2, 40]),
    (100, 14, 2, [99, 100, 101, 350]),
    (48, 8, 2, [47, 48, 49, 500]),
])
def test_decode_matches_plain(cuda_lib, bs, hq, hkv, lens):
    pa = cuda_lib
    c = _case(pa, lens, bs, hq, hkv, seed=len(lens) + bs)
    out = _decode(pa, c)
    _check_decode(out, c)
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any()
    assert pa.device_errors() == 0


# Shares long enough that a pair's beginning counts: many pairs a CTA, empty and one-token
# sequences between them, and a few pairs that many CTAs share.
@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (16, 16, 8, [(i * 389) % 601 for i in range(33)] + [0, 0, 1, 1, 2, 0, 599, 0]),
    (48, 8, 8, [(i * 577) % 1201 for i in range(34)] + [1, 0]),
    (64, 16, 4, [0, 20001, 0]),
    (832, 8, 2, [15000, 1, 30000, 33]),
])
def test_decode_long_shares(cuda_lib, bs, hq, hkv, lens):
    c = _case(cuda_lib, lens, bs, hq, hkv, seed=bs)
    _check_decode(_decode(cuda_lib, c), c)
    assert cuda_lib.device_errors() == 0


# Clusters of 1 to 16 CTAs, parts without a tile, empty sequences beside others, lengths at the ends of
# tiles and pages and of what a cluster takes.
@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (16, 8, 1, [1]), (16, 8, 1, [64]), (16, 6, 1, [65]), (64, 8, 2, [128, 0, 1]), (832, 24, 4, [1024]),
    (832, 24, 4, [1025, 3]), (64, 24, 4, [1536]), (64, 24, 4, [1537]), (7, 7, 1, [130, 7, 0, 8, 64]),
    (100, 3, 3, [257, 256, 255]), (16, 64, 8, [500, 499]), (48, 12, 4, [0, 700]),
    (64, 16, 4, [(i * 37) % 130 for i in range(19)]), (16, 300, 300, [5]), (1, 2, 2, [33, 17]),
])
def test_decode_short_sequences(cuda_lib, bs, hq, hkv, lens):
    pa = cuda_lib
    c = _case(pa, lens, bs, hq, hkv, seed=bs + len(lens))
    out = _decode(pa, c)
    _check_decode(out, c)
    assert torch.equal(out, _decode(pa, c))
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any()
    assert pa.device_errors() == 0


# One sequence, whose pairs are cut by themselves: from a tile to one part a CTA of the GPU, and more
# KV heads than fit; and more sequences than a warp keeps the lengths of.
@pytest.mark.parametrize("bs,hq,hkv,lens", [
    (16, 5, 1, [20001]), (832, 8, 1, [40000]), (64, 16, 16, [130]), (16, 320, 320, [37]), (7, 64, 32, [100]),
    (16, 4, 1, [(i * 61) % 97 for i in range(131)]), (64, 8, 2, [(i * 61) % 301 for i in range(200)]),
    (16, 2, 2, [(i * 7) % 40 for i in range(128)]),
])
def test_decode_one_sequence_and_many(cuda_lib, bs, hq, hkv, lens):
    c = _case(cuda_lib, lens, bs, hq, hkv, seed=bs)
    _check_decode(_decode(cuda_lib, c), c)
    assert cuda_lib.device_errors() == 0


def test_decode_longest_length_of_a_short_sequence(cuda_lib):
    # One sequence of 100 keys whose table has room for 2^31 - 1: no error.
    pa = cuda_lib
    bs, hkv = 1 << 16, 16
    codes, scales = pa.q8_cache_shapes(1, bs, hkv)
    cache = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (codes, codes, scales, scales)]
    cache[:2] = [c.view(torch.float8_e4m3fn) for c in cache[:2]]
    table = torch.zeros(1, 1 << 15, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, 256, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(100, hkv, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    pa.reshape_and_cache_q8(k, v, *cache, torch.arange(100, device="cuda"))
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    out = pa.decode_q8(q, *cache, table, lens, 0.0625, 2**31 - 1)
    assert pa.device_errors() == 0
    # (as many CTAs as the length allows, so other parts, whose sums may round a result to the next
    # BF16 value: 2^-7 of it at most)
    want = pa.decode_q8(q, *cache, table, lens, 0.0625, 100)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()


@pytest.mark.parametrize("S", [1, 4, 40])
def test_decode_of_lengths_that_the_kernel_before_writes(cuda_lib, S):
    # The decode looks at lengths and tables before the preparation that writes them has ended.
    pa = cuda_lib
    c = _case(pa, [900] * S, 64, 24, 4, seed=5)
    free = torch.zeros(S * 20, dtype=torch.int32, device="cuda")
    new = torch.ones(S, dtype=torch.int32, device="cuda")
    steps, prep = [], None
    for i in range(12):
        # (odd: no sequence begins a page, which the preparation would take from the free list)
        computed = torch.tensor([(j * 131 + i * 377) % 899 | 1 for j in range(S)], dtype=torch.int32, device="cuda")
        tables = c["bt"][torch.randperm(S, generator=torch.Generator().manual_seed(i))].contiguous()
        steps.append((computed, tables))
    bt = c["bt"].clone()
    ws = torch.empty(pa.decode_q8_workspace_size(S, 24, 4, 256, 64, 900), dtype=torch.uint8, device="cuda")
    outs = []
    for computed, tables in steps:
        pa.copy(bt, tables) if bt.numel() * 4 % 16 == 0 else bt.copy_(tables)
        prep = pa.batch_input_prep(computed, new, [bt], [64], [free], S, out=prep)
        outs.append(pa.decode_q8(c["q"], *c["cache"], bt, prep["seq_lens"], 0.0625, 900, workspace=ws))
    torch.cuda.synchronize()
    for (computed, tables), out in zip(steps, outs):
        assert torch.equal(out, pa.decode_q8(c["q"], *c["cache"], tables, computed + 1, 0.0625, 900))
        torch.cuda.synchronize()
    assert pa.device_errors() == 0


@pytest.mark.parametrize("S,n", [(1, 5000), (1, 200), (3, 260), (24, 2000)])
def test_decode_of_a_table_that_the_kernel_before_writes(cuda_lib, S, n):
    # What the decode looks at before that kernel ends: valid pages, but of other sequences, entries
    # outside the pool, other lengths.
    pa = cuda_lib
    c = _case(pa, [n] * (S + 2), 16, 12, 2, seed=S)
    width = c["bt"].shape[1] // 4 * 4  # (copies of whole 16 bytes)
    most = width * 16
    bt = torch.zeros(S, width, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S + 3 & ~3, dtype=torch.int32, device="cuda")
    steps = []
    for i in range(16):
        pick = torch.randperm(S + 2, generator=torch.Generator().manual_seed(i))[:S]
        table = c["bt"][pick, :width].contiguous()
        count = torch.full_like(lens, most if i % 4 < 3 else most - 70 - i)
        if i % 5 == 4:
            count[0], table[0] = 0, -7  # no keys: its entries are not looked at
        steps.append((table, count))
    ws = torch.empty(pa.decode_q8_workspace_size(S, 12, 2, 256, 16, most), dtype=torch.uint8, device="cuda")
    outs = []
    for table, count in steps:
        pa.copy(lens, count)
        pa.copy(bt, table)
        outs.append(pa.decode_q8(c["q"][:S], *c["cache"], bt, lens[:S], 0.0625, most, workspace=ws))
    for table, count in steps:
        pa.copy(bt, table)
        pa.copy(lens, count)
        outs.append(pa.decode_q8(c["q"][:S], *c["cache"], bt, lens[:S], 0.0625, most, workspace=ws))
    torch.cuda.synchronize()
    for (table, count), *got in zip(steps, outs[:16], outs[16:]):
        want = pa.decode_q8(c["q"][:S], *c["cache"], table, count[:S], 0.0625, most)
        assert torch.equal(got[0], want) and torch.equal(got[1], want)
        torch.cuda.synchronize()
    assert pa.device_errors() == 0


def test_steps_of_write_and_decode_back_to_back(cuda_lib):
    # Each step's write grows scales that the step before has read: no stale ones are used.
    pa = cuda_lib
    S, bs, hkv, start, steps = 6, 64, 4, 700, 40
    c = _case(pa, [start + steps] * S, bs, 24, hkv, seed=6)
    plain = [x.clone() for x in c["cache"]]
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.arange(S, device="cuda") * (start + steps) + start
    lens = [torch.full((S,), start + i + 1, dtype=torch.int32, device="cuda") for i in range(steps)]
    slots = [c["slots"][rows + i].contiguous() for i in range(steps)]
    kv = [[(torch.randn(S, hkv, 256, generator=g, device="cuda") * 2.0 ** (i % 16)).to(torch.bfloat16)
           for _ in range(2)] for i in range(steps)]
    ws = torch.empty(pa.decode_q8_workspace_size(S, 24, hkv, 256, bs, start + steps), dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(steps):
        pa.reshape_and_cache_q8(*kv[i], *c["cache"], slots[i])
        outs.append(pa.decode_q8(c["q"], *c["cache"], c["bt"], lens[i], 0.0625, start + steps, workspace=ws))
    torch.cuda.synchronize()
    for i in range(steps):
        pa.reshape_and_cache_q8(*kv[i], *plain, slots[i])
        torch.cuda.synchronize()
        assert torch.equal(outs[i], pa.decode_q8(c["q"], *plain, c["bt"], lens[i], 0.0625, start + steps)), i
        torch.cuda.synchronize()
    for a, b in zip(c["cache"], plain):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_decode_scales(cuda_lib, scale):
    c = _case(cuda_lib, [300, 17], 64, 6, 1, seed=9)
    _check_decode(_decode(cuda_lib, c, scale), c, scale)


@pytest.mark.parametrize("q,k,v", [(1e-3, 1e3, 1e-20), (1e4, 1e-4, 1e20), (1e30, 1e-30, 1.0),
                                   (1e-30, 1.0, 3e4), (1e-30, 1e30, 1e-28), (1.0, 1e-36, 1e28)])
def test_decode_magnitudes(cuda_lib, q, k, v):
    c = _case(cuda_lib, [700], 64, 6, 1, seed=4, scale_k=k, scale_v=v)
    c["q"] = (c["q"].float() * q).to(torch.bfloat16)
    _check_decode(_decode(cuda_lib, c), c)


def _refill(pa, c, k, v):
    for x in c["cache"]:
        x.view(torch.uint8).fill_(0xFF)
    pa.reshape_and_cache_q8(_bf(k), _bf(v), *c["cache"], c["slots"])


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("at", [0, 250, 499])
def test_decode_large_values_of_negligible_weight(cuda_lib, size, at):
    # One block of V is `size` times as large as the others, its tokens' weights e^-60 times as large
    # (and, for the smaller sizes, without part in the result): the others keep their bits.
    pa = cuda_lib
    c = _case(pa, [500], 64, 6, 1, seed=11)
    rng = np.random.default_rng(3)
    q = rng.standard_normal(256)
    c["q"] = _bf(np.broadcast_to(q, (1, 6, 256)))
    k, v = rng.standard_normal((500, 1, 256)), rng.standard_normal((500, 1, 256))
    b = at // 16 * 16
    k[b:b + 16] -= q * (60 / 0.0625 / (q @ q))
    v[b:b + 16] *= size
    _refill(pa, c, k, v)
    _check_decode(_decode(pa, c), c)


def test_decode_scores_that_grow_along_the_keys(cuda_lib):
    # The references move at every tile, V's scales up and down beside them.
    pa = cuda_lib
    c = _case(pa, [2000], 64, 8, 1, seed=12)
    rng = np.random.default_rng(5)
    q = rng.standard_normal(256)
    c["q"] = _bf(np.broadcast_to(q, (1, 8, 256)))
    k, v = rng.standard_normal((2000, 1, 256)), rng.standard_normal((2000, 1, 256))
    k += (np.arange(2000) / 2000 * 300)[:, None, None] * q / 0.0625 / (q @ q)
    v *= 2.0 ** rng.integers(-20, 20, (125,)).repeat(16)[:, None, None]
    _refill(pa, c, k, v)
    _check_decode(_decode(pa, c), c)


@pytest.mark.parametrize("bs,hq,hkv,lens", [(64, 8, 1, [500]), (16, 16, 2, [4096, 40]), (832, 24, 4, [9000])])
def test_decode_flat_scores_count_every_token(cuda_lib, bs, hq, hkv, lens):
    # q = 0 and one-hot values: dim d of the output is how many tokens have it, over all.
    pa = cuda_lib
    c = _case(pa, lens, bs, hq, hkv, seed=13)
    c["q"].zero_()
    N = sum(lens)
    v = np.zeros((N, hkv, 256))
    d = np.random.default_rng(1).integers(0, 256, (N, hkv))
    np.put_along_axis(v, d[..., None], 1.0, 2)
    _refill(pa, c, np.zeros_like(v), v)
    out, first = f64(_decode(pa, c)), 0
    for s, n in enumerate(lens):
        for h in range(hq):
            count = np.bincount(d[first:first + n, h // (hq // hkv)], minlength=256) / n
            assert (np.abs(out[s, h] - count) <= count * (2.0 ** -8 + 2.0 ** -12)).all()
        first += n


@pytest.mark.parametrize("scale_v", [1e-28, 1.0, 1e28])
def test_decode_of_one_token_is_its_row(cuda_lib, scale_v):
    pa = cuda_lib
    c = _case(pa, [1, 1, 1], 16, 16, 2, seed=14, scale_v=scale_v)
    out = _decode(pa, c)
    want = pa.gather_cache_q8(*c["cache"], c["slots"])[1]
    assert torch.equal(out, want.repeat_interleave(8, 1))


@pytest.mark.parametrize("n,at", [(3000, 0), (3000, 1777), (3000, 2999), (40, 20), (9000, 8190)])
def test_decode_of_a_token_that_outweighs_the_others_is_its_row(cuda_lib, n, at):
    pa = cuda_lib
    c = _case(pa, [n], 64, 8, 2, seed=15)
    q = torch.randn(256, generator=torch.Generator().manual_seed(1))
    c["q"] = _bf(q.expand(1, 8, 256))
    k = torch.randn(n, 2, 256, generator=torch.Generator().manual_seed(2)) * 0.1
    k[at] += q * (300 / 0.0625 / float(q @ q))
    v = torch.randn(n, 2, 256, generator=torch.Generator().manual_seed(3))
    _refill(pa, c, k, v)
    out = _decode(pa, c)
    want = pa.gather_cache_q8(*c["cache"], c["slots"][at:at + 1])[1]
    assert torch.equal(out, want.repeat_interleave(4, 1))


def test_decode_nan_reaches_its_head_and_nothing_else(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [300, 200, 9000], 64, 6, 3, seed=16)
    clean = _decode(pa, c)
    kc, vc, ks, vs = c["cache"]
    kb, vb = kc.view(torch.uint8), vc.view(torch.uint8)
    page = lambda s, t: int(c["table"][s, t // 64])
    kb[page(0, 130), 130 % 64, 1, 9] = 0x7F     # a key: its head, of its sequence
    vb[page(1, 70), 70 % 64, 2, 17] = 0xFF      # a value: one dim
    ks[page(2, 8000), 8000 % 64 // 16, 0] = 255  # a block's scale
    out = _decode(pa, c)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, 2:4] = True
    nan[1, 4:6, 17] = True
    nan[2, 0:2] = True
    assert torch.equal(torch.isnan(out), nan) and torch.equal(out[~nan], clean[~nan])
    ks[page(2, 8000), 8000 % 64 // 16, 0] = 120
    vs[page(2, 77), 77 % 64 // 16, 1] = 255
    out = _decode(pa, c)
    assert torch.isnan(out[2, 2:4]).all() and not torch.isnan(out[2, :2]).any() and not torch.isnan(out[2, 4:]).any()


def test_decode_nan_value_of_vanishing_weight(cuda_lib):
    # The first keys outweigh the rest by e^200: the NaN is in another part, of weight 0 in fp32.
    pa = cuda_lib
    c = _case(pa, [9000], 64, 8, 2, seed=1)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(256, generator=g)
    c["q"] = _bf(q.expand(1, 8, 256))
    x, y = torch.randn(9000, 2, 256, generator=g), torch.randn(9000, 2, 256, generator=g)
    x[:8] += (q * (200 / 0.0625 / float(q @ q)))[None, None]
    _refill(pa, c, x, y)
    fine = c["cache"][1].view(torch.uint8).clone()
    for at in range(100, 9000, 900):
        codes = c["cache"][1].view(torch.uint8)
        codes.copy_(fine)
        codes[int(c["table"][0, at // 64]), at % 64, 1, 70] = 0x7F
        nan = torch.isnan(_decode(pa, c)[0])
        assert nan[4:, 70].all() and int(nan.sum()) == 4, at


def test_decode_bad_pages_and_lengths_are_reported(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [200, 300, 100], 64, 6, 1, seed=17)
    good = _decode(pa, c)
    bt = c["bt"].clone()
    for bad in (-1, -(2**31), c["cache"][0].shape[0], 2**31 - 1):
        bt[0, 1] = bad
        out = pa.decode_q8(c["q"], *c["cache"], bt, c["lens"], 0.0625, 300)
        assert pa.device_errors() == pa.DEVERR_PAGE
        assert torch.equal(out[1:], good[1:])
        # the page's 64 tokens are zeros: scores 0, values 0
        zc = [x.clone() for x in c["cache"]]
        page = int(c["table"][0, 1])
        zc[0].view(torch.uint8)[page] = 0
        zc[1].view(torch.uint8)[page] = 0
        zc[2][page] = zc[3][page] = 127
        assert torch.equal(out[0], _decode(pa, dict(c, cache=zc))[0])
    lens = c["lens"].clone()
    lens[1], lens[2] = 301, -4
    out = pa.decode_q8(c["q"], *c["cache"], c["bt"], lens, 0.0625, 300)
    assert pa.device_errors() == pa.DEVERR_SEQLEN
    assert torch.equal(out[:2], good[:2]) and not out[2].any()


def test_decode_table_wider_than_needed_and_strided(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [200, 300], 64, 6, 1, seed=18)
    wide = torch.full((2, 40), -7, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + c["bt"].shape[1]] = c["bt"]
    q = torch.randn(2, 18, 256, device="cuda").to(torch.bfloat16)[:, 6:12]
    out = pa.decode_q8(q, *c["cache"], wide[:, 3:], c["lens"], 0.0625, 300)
    assert torch.equal(out, pa.decode_q8(q.contiguous(), *c["cache"], c["bt"], c["lens"], 0.0625, 320))


def test_decode_deterministic_dirty_workspace_and_stream(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [5000, 0, 77, 3000], 64, 24, 4, seed=19)
    need = pa.decode_q8_workspace_size(4, 24, 4, 256, 64, 5000)
    first = _decode(pa, c)
    side = torch.cuda.Stream()
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = _decode(pa, c, workspace=ws)
        side.synchronize()
        assert torch.equal(out, first)
    with pytest.raises(pa.PAError):
        _decode(pa, c, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_write_and_decode_in_two_graphs_with_their_own_workspaces(cuda_lib):
    pa = cuda_lib
    cases = [_case(pa, lens, 64, 24, 4, seed=20 + i) for i, lens in enumerate(([3000, 5], [40, 900]))]
    plans = []
    for c in cases:
        S, most = len(c["lens"]), int(c["lens"].max())
        ends = torch.cumsum(c["lens"], 0).long() - 1
        slots = c["slots"][ends].contiguous()  # each sequence's newest token comes again in the step
        k, v = (torch.randn(S, 4, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
        ws = torch.empty(pa.decode_q8_workspace_size(S, 24, 4, 256, 64, most), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c["q"])

        def step(c=c, k=k, v=v, slots=slots, ws=ws, out=out, most=most):
            pa.reshape_and_cache_q8(k, v, *c["cache"], slots)
            pa.decode_q8(c["q"], *c["cache"], c["bt"], c["lens"], 0.0625, most, out=out, workspace=ws)

        step()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        plans.append((graph, out, want, step))  # (step holds the tensors that the graph reads)
    for _ in range(3):
        for graph, out, want, _step in plans:
            out.fill_(9.0)
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, want, _step in plans:
            assert torch.equal(out, want)
    assert pa.device_errors() == 0


def test_offsets_past_32_bits(cuda_lib):
    # Pages 64 MB apart, the used ones past 4 GB.
    pa = cuda_lib
    pages, bs, hkv = 80, 16, 1
    stride = 64 << 20
    store = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    kc = store.as_strided((pages, bs, hkv, 256), (stride, hkv * 256, 256, 1)).view(torch.float8_e4m3fn)
    vc = store[1 << 20:].as_strided((pages, bs, hkv, 256), (stride, hkv * 256, 256, 1)).view(torch.float8_e4m3fn)
    ks = store[2 << 20:].as_strided((pages, 1, hkv), (stride // 2, hkv, 1))
    vs = store[3 << 20:].as_strided((pages, 1, hkv), (stride // 2, hkv, 1))
    small = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (*pa.q8_cache_shapes(4, bs, hkv),) * 2]
    small = [small[0].view(torch.float8_e4m3fn), small[2].view(torch.float8_e4m3fn), small[1], small[3]]
    n = 60
    t = torch.arange(n, device="cuda")
    k, v = (torch.randn(n, hkv, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    page = torch.tensor([79, 65, 70, 78], dtype=torch.int32, device="cuda")
    pa.reshape_and_cache_q8(k, v, kc, vc, ks, vs, page.long()[t // bs] * bs + t % bs)
    pa.reshape_and_cache_q8(k, v, *small, t)
    q = torch.randn(3, 4, 256, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    few = torch.arange(4, dtype=torch.int32, device="cuda")
    assert torch.equal(pa.decode_q8(q[:1], kc, vc, ks, vs, page[None], lens, 0.0625, n),
                       pa.decode_q8(q[:1], *small, few[None], lens, 0.0625, n))
    assert torch.equal(pa.prefill_chunk_q8(q, kc, vc, ks, vs, page, n - 3, True, 0.0625),
                       pa.prefill_chunk_q8(q, *small, few, n - 3, True, 0.0625))
    a = pa.gather_cache_q8(kc, vc, ks, vs, page.long()[t // bs] * bs + t % bs)
    b = pa.gather_cache_q8(*small, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert pa.device_errors() == 0


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0] * 40])
@pytest.mark.parametrize("max_len", [1, 100, 9000])
def test_decode_of_padding_entries_alone(cuda_lib, lens, max_len):
    pa = cuda_lib
    c = _case(pa, [64], 64, 8, 2, seed=3)
    S = len(lens)
    q = torch.randn(S, 8, 256, device="cuda").to(torch.bfloat16)
    need = pa.decode_q8_workspace_size(S, 8, 2, 256, 64, max_len)
    for fill in (0, 0xFF):
        out = torch.full_like(q, 3.0)
        pa.decode_q8(q, *c["cache"], torch.full((S, 141), -1, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.0625, max_len, out=out,
                     workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        assert not out.any()
    assert pa.device_errors() == 0


# ------------------------------------------------------------------------------ prefill
def _check_prefill(got, c, cu, lens, causal=True, scale=0.0625):
    ref, tol = _q8.prefill(f64(c["q"]), *_plain_caches(c), c["table"], cu, lens, causal, scale)
    d = np.abs(f64(got) - ref)
    assert np.isfinite(d).all()
    assert (d <= tol).all(), (d.max(), (d / tol).max())


@pytest.mark.parametrize("q_len,q_start,bs,hq,hkv,causal", [
    (1, 0, 16, 4, 1, True), (1, 4000, 832, 24, 4, True), (130, 900, 832, 24, 4, True),
    (128, 0, 64, 6, 1, False), (300, 77, 7, 8, 2, True), (257, 1000, 784, 10, 2, False),
    (40, 3000, 48, 5, 5, True), (2, 255, 1, 3, 1, True), (513, 0, 100, 2, 2, True),
    (3, 16384, 64, 4, 2, True), (3, 16381, 7, 4, 2, True), (2, 40001, 20, 2, 1, False),
])
def test_prefill_chunk_matches_plain(cuda_lib, q_len, q_start, bs, hq, hkv, causal):
    pa = cuda_lib
    n = q_start + q_len
    c = _case(pa, [n], bs, hq, hkv, seed=n, rows=q_len)
    out = pa.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], q_start, causal, 0.0625)
    _check_prefill(out, c, [0, q_len], [n], causal)
    assert pa.device_errors() == 0


def test_prefill_varlen_over_two_launches_and_empty_chunks(cuda_lib):
    pa = cuda_lib
    rows = [(i * 37) % 60 for i in range(40)]
    lens = [r + (i * 53) % 400 if r else 0 for i, r in enumerate(rows)]
    lens = [max(n, 1) for n in lens]
    cu = np.concatenate([[0], np.cumsum(rows)]).tolist()
    c = _case(pa, lens, 16, 8, 2, seed=30, rows=cu[-1])
    out = pa.prefill_varlen_q8(c["q"], *c["cache"], c["bt"], cu, lens, True, 0.0625)
    _check_prefill(out, c, cu, lens)
    assert pa.device_errors() == 0


def test_prefill_split_items_and_less_workspace(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [9000], 832, 24, 4, seed=31, rows=20)
    args = (c["q"], *c["cache"], c["bt"], [0, 20], [9000], True, 0.0625)
    need = pa.prefill_varlen_q8_workspace_size([0, 20], [9000], True, 24, 4, 256, 832)
    out = pa.prefill_varlen_q8(*args)
    _check_prefill(out, c, [0, 20], [9000])
    for fill in (0, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(pa.prefill_varlen_q8(*args, workspace=ws), out)
    with pytest.raises(pa.PAError):
        pa.prefill_varlen_q8(*args, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("q,k,v", [(1e-3, 1e3, 1e-20), (1e4, 1e-4, 1e20), (1e20, 1e-20, 1e-6)])
def test_prefill_magnitudes(cuda_lib, q, k, v):
    c = _case(cuda_lib, [400], 64, 6, 1, seed=32, rows=100, scale_k=k, scale_v=v)
    c["q"] = (c["q"].float() * q).to(torch.bfloat16)
    out = cuda_lib.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], 300, True, 0.0625)
    _check_prefill(out, c, [0, 100], [400])


@pytest.mark.parametrize("apart", [2.0 ** 4, 2.0 ** 9, 2.0 ** 14])
def test_prefill_uneven_blocks(cuda_lib, apart):
    # Scales of V's and K's blocks up to `apart` either way: still exact operands.  (The weights keep
    # their bits relative to the row's largest, whatever V's sizes are.)
    pa = cuda_lib
    c = _case(pa, [500], 64, 6, 2, seed=33, rows=60)
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((500, 2, 256)), rng.standard_normal((500, 2, 256))
    v[100:116] *= apart
    v[200:300] /= apart ** 0.5
    k[320:340] /= apart
    _refill(pa, c, k, v)
    out = pa.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], 440, True, 0.0625)
    _check_prefill(out, c, [0, 60], [500])


def test_prefill_far_smaller_blocks(cuda_lib):
    # V of head 0 is 2^-40 of one block's: that block loses its bits, not the others; where no row
    # sees the block, what is off is at most 2^-39 of its largest value.
    pa = cuda_lib
    c = _case(pa, [64], 16, 2, 1, seed=34, rows=32)
    rng = np.random.default_rng(2)
    v = rng.standard_normal((64, 1, 256))
    v[48:] *= 2.0 ** 40
    _refill(pa, c, rng.standard_normal((64, 1, 256)), v)
    out = pa.prefill_chunk_q8(c["q"], *c["cache"], c["bt"][0], 32, True, 0.0625)
    ref, tol = _q8.prefill(f64(c["q"]), *_plain_caches(c), c["table"], [0, 32], [64], True, 0.0625)
    assert (np.abs(f64(out) - ref) <= tol + 2.0 ** -39 * np.abs(v).max()).all()


def test_prefill_nan_key_bad_page_and_graph(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [300], 64, 6, 2, seed=35, rows=100)
    args = (c["q"], *c["cache"], c["bt"], [0, 100], [300], True, 0.0625)
    ws = torch.empty(pa.prefill_varlen_q8_workspace_size([0, 100], [300], True, 6, 2, 256, 64),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c["q"])
    pa.prefill_varlen_q8(*args, workspace=ws, out=out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.prefill_varlen_q8(*args, workspace=ws, out=out)
    out.zero_()
    ws.fill_(0xFF)
    graph.replay()
    assert torch.equal(out, want)
    codes = c["cache"][0].view(torch.uint8)
    page = int(c["table"][0, 250 // 64])
    keep = int(codes[page, 250 % 64, 1, 0])
    codes[page, 250 % 64, 1, 0] = 0x7F  # row 50 and later, heads 3 ..
    got = pa.prefill_varlen_q8(*args)
    assert torch.isnan(got[50:, 3:]).all() and torch.equal(got[:, :3], want[:, :3])
    assert torch.equal(got[:50, 3:], want[:50, 3:])
    codes[page, 250 % 64, 1, 0] = keep
    assert pa.device_errors() == 0
    bt = c["bt"].clone()
    bt[0, 0] = -3
    pa.prefill_varlen_q8(c["q"], *c["cache"], bt, [0, 100], [300], True, 0.0625)
    assert pa.device_errors() == pa.DEVERR_PAGE


class _Nothing:
    """In the place of the short calls: takes none."""

    def __getattr__(self, name):
        return lambda *a: None


def test_short_calls_are_the_others(cuda_lib, monkeypatch):
    # What the compiled module takes gives what the Python checks and ctypes give, and what it leaves
    # to them is taken: other number types, one page, one token, a row of the table, given outputs.
    pa = cuda_lib
    c = _case(pa, [300, 77], 64, 24, 4, seed=40)
    k, v = (torch.randn(77, 4, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    cs = torch.randn(100, 64, device="cuda")
    w = torch.randn(256, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 100, (3, 77), device="cuda", dtype=torch.int32)
    q = torch.randn(77, 24, 256, device="cuda").to(torch.bfloat16)
    axes = pa.mrope_axes([16, 8, 8])
    slots = c["slots"][300:].contiguous()

    def calls():
        cache = [x.clone() for x in c["cache"]]
        got = [pa.reshape_and_cache_q8(k, v, *cache, slots)] + cache
        got += pa.gather_cache_q8(*cache, slots)
        got.append(pa.decode_q8(c["q"], *cache, c["bt"], c["lens"], 0.0625, 300))
        out, ws = torch.empty_like(c["q"]), torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        assert pa.decode_q8(c["q"], *cache, c["bt"], c["lens"], 0.0625, 300, out, ws) is out
        got += [out, pa.decode_q8(c["q"][:1], *cache, c["bt"][:1], c["lens"][:1], 1, np.int64(300))]
        for how in (dict(), dict(out=torch.empty_like(c["q"]), workspace=ws)):
            got.append(pa.prefill_varlen_q8(c["q"], *cache, c["bt"], [0, 1, 2], [300, 77], True, 0.0625, **how))
        got.append(pa.prefill_chunk_q8(c["q"], *cache, c["bt"][0], 200, False, 0.0625))
        got.append(pa.prefill_varlen_q8(c["q"], *cache, c["bt"], np.array([0, 1, 2]), (300, 77), 1, 0.0625))
        got += pa.qk_norm_mrope(q, k, w, w, cs, pos, axes, 1e-6)
        got += pa.qk_norm_mrope(q, k, w, w, cs, pos, list(axes), np.float32(1e-6), 1, 0)
        bf = torch.zeros(2, 2, 64, 4, 256, dtype=torch.bfloat16, device="cuda")
        at = torch.arange(77, device="cuda")
        got.append(pa.qk_norm_mrope_cache(q, k, v, w, w, cs, pos, axes, 1e-6, bf[:, 0], bf[:, 1], at))
        one = [x[:1] for x in cache]
        got += [bf] + list(pa.gather_cache_q8(*one, at[:1])) + list(pa.gather_cache_q8(*one, at[:0]))
        return [x if x is None else x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in got]

    short = calls()
    monkeypatch.setattr(pa, "_bind", _Nothing())
    for a, b in zip(short, calls(), strict=True):
        assert a is b is None or torch.equal(a, b)
    monkeypatch.undo()
    for bind in (pa._bind, _Nothing()):
        monkeypatch.setattr(pa, "_bind", bind)
        with pytest.raises(pa.PAError):  # refused by the library either way
            pa.reshape_and_cache_q8(k, v, c["cache"][0], c["cache"][0], *c["cache"][2:], slots)
        with pytest.raises(pa.PAError):
            pa.decode_q8(c["q"], *c["cache"], c["bt"], c["lens"], float("inf"), 300)
        with pytest.raises(pa.PAError):
            pa.prefill_varlen_q8(c["q"], *c["cache"], c["bt"], [0, 2, 2], [1, 77], True, 0.0625)
    assert pa.device_errors() == 0


def test_layout_refusals(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [100], 16, 6, 2, seed=36)
    kc, vc, ks, vs = c["cache"]
    q, bt, lens = c["q"], c["bt"], c["lens"]
    for bad in ((kc.view(torch.uint8), vc, ks, vs), (kc, vc, ks.float(), vs)):
        with pytest.raises(TypeError):
            pa.decode_q8(q, *bad, bt, lens, 0.0625, 100)
    for bad in ((kc[:-1], vc, ks, vs), (kc, vc, ks[:-1], vs[:-1]), (kc, vc, ks[:, :, :1], vs[:, :, :1]),
                (kc[:, :, :1], vc[:, :, :1], ks, vs), (kc.transpose(1, 2), vc.transpose(1, 2), ks, vs)):
        with pytest.raises(ValueError):
            pa.decode_q8(q, *bad, bt, lens, 0.0625, 100)
    with pytest.raises(ValueError):
        pa.decode_q8(q, kc, vc, ks, vs, bt, lens, 0.0625, 200)  # the table has room for 112
    with pytest.raises(ValueError):
        pa.decode_q8(q, kc, vc, ks, vs, bt, lens, 0.0625, 2**32 + 100)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_q8(q[:, :2], q[:, :1], kc, vc, ks, vs, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pa.gather_cache_q8(kc, vc, ks, vs, torch.zeros(4, dtype=torch.int64, device="cuda")[::2])
    with pytest.raises(ValueError):
        pa.prefill_varlen_q8(q, kc, vc, ks, vs, bt, [0, 2], [100], True, 0.0625)
    with pytest.raises(pa.PAError):
        pa.prefill_chunk_q8(q, kc, vc, ks, vs, bt[0], -1, True, 0.0625)
