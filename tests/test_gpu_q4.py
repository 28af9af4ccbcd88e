"""The 4-bit cache on the GPU: writes and reads bit for bit, decode and prefill against the
plain 64-bit attention over the values the cache stands for."""
import numpy as np
import pytest
import torch

import _q4

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # half a BF16 step, relative


def _bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _rows(T, hkv, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, 256, generator=g)
    if kind == "outliers":
        x[:, :, ::37] *= 60
    elif kind == "constant":
        x[:] = torch.randn(T, hkv, 1, generator=g)
    elif kind == "integers":  # many ties: quarters of small integers
        x = torch.randint(-30, 31, x.shape, generator=g) / 4.0
    elif kind == "tiny":
        x *= 1e-38
    elif kind == "huge":
        x *= 1e37
    elif kind == "offset":
        x = x * 1e-6 + torch.randint(0, 2, x.shape, generator=g) - 0.5
    return x.to(torch.bfloat16)


def _same_cache(got, want, msg=""):
    assert np.array_equal(got.cpu().numpy(), want), msg


@pytest.mark.parametrize("kind", ["normal", "outliers", "constant", "integers", "tiny", "huge",
                                  "offset"])
@pytest.mark.parametrize("bs,hkv,T", [(16, 4, 9), (1, 1, 3), (7, 2, 16)])
def test_write_matches_plain_bits(cuda_lib, kind, bs, hkv, T):
    pa = cuda_lib
    key, val = _rows(T, hkv, 1, kind), _rows(T, hkv, 2, kind)
    pages = -(-T // bs) + 2
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(pages * bs, generator=g)[:T]
    kc = torch.full(pa.q4_cache_shape(pages, bs, hkv), 0xA5, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    want = [_q4.empty_cache(pages, bs, hkv, 0xA5) for _ in range(2)]
    for x, c in zip((key, val), want):
        n, s, lo = _q4.quantise(_q4.f64(x))
        for t in range(T):
            for h in range(hkv):
                _q4.store(c, bs, int(slots[t]), h, n[t, h], s[t, h], lo[t, h])
    pa.reshape_and_cache_q4(key.cuda(), val.cuda(), kc, vc, slots.cuda())
    _same_cache(kc, want[0], "K")
    _same_cache(vc, want[1], "V")
    ko, vo = pa.gather_cache_q4(kc, vc, slots.cuda())
    for got, x in ((ko, key), (vo, val)):
        n, s, lo = _q4.quantise(_q4.f64(x))
        v = _q4.value(n, s, lo)
        # one rounding in fp32 (of lo + s n), one to BF16 (subnormal step: 2^-133)
        tol = np.abs(v) * HALF * 1.01 + (np.abs(lo) + 15 * s).repeat(64, -1).reshape(v.shape) * 2.0 ** -24 + 2.0 ** -134
        assert (np.abs(_q4.f64(got) - v) <= tol).all()
    assert pa.device_errors() == 0


def test_write_non_finite_groups_read_back_as_nan(cuda_lib):
    pa = cuda_lib
    x = _rows(3, 1, 5)
    x[0, 0, 3] = float("nan")
    x[1, 0, 70] = float("inf")
    x[2, 0, 130], x[2, 0, 131] = 3e38, -3e38  # a range past fp32
    kc = torch.zeros(pa.q4_cache_shape(1, 16, 1), dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    slots = torch.tensor([4, 0, 9], device="cuda")
    pa.reshape_and_cache_q4(x.cuda(), x.cuda(), kc, vc, slots)
    ko, vo = pa.gather_cache_q4(kc, vc, slots)
    bad = np.zeros((3, 256), bool)
    bad[0, :64] = bad[1, 64:128] = bad[2, 128:192] = True
    for o in (ko, vo):
        assert np.array_equal(np.isnan(_q4.f64(o)[:, 0]), bad)


def test_write_and_gather_padding_bounds_and_strides(cuda_lib):
    pa = cuda_lib
    T, hkv, bs, pages = 6, 2, 16, 3
    packed = torch.randn(T, 3 * hkv * 256, device="cuda").to(torch.bfloat16)
    key = packed[:, hkv * 256:2 * hkv * 256].unflatten(1, (hkv, 256))
    val = packed[:, 2 * hkv * 256:].unflatten(1, (hkv, 256))
    both = torch.zeros((pages, 2) + pa.q4_cache_shape(1, bs, hkv)[1:], dtype=torch.uint8, device="cuda")
    kc, vc = both.unbind(1)  # pages twice as far apart
    slots = torch.tensor([5, -1, 47, -7, 30, pages * bs], device="cuda")
    pa.reshape_and_cache_q4(key, val, kc, vc, slots)
    assert pa.device_errors() == pa.DEVERR_SLOT
    plain_k = torch.zeros(pa.q4_cache_shape(pages, bs, hkv), dtype=torch.uint8, device="cuda")
    plain_v = plain_k.clone()
    ok = torch.tensor([0, 2, 4], device="cuda")
    pa.reshape_and_cache_q4(key[ok], val[ok], plain_k, plain_v, slots[ok])
    assert torch.equal(kc, plain_k) and torch.equal(vc, plain_v)
    ko = torch.full((T, hkv, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    pa.gather_cache_q4(kc, vc, slots, ko, vo)
    assert pa.device_errors() == pa.DEVERR_SLOT
    assert not ko[[1, 3, 5]].any() and not vo[[1, 3, 5]].any()
    k1, v1 = pa.gather_cache_q4(plain_k, plain_v, slots[ok])
    assert torch.equal(ko[ok], k1) and torch.equal(vo[ok], v1)
    pa.reshape_and_cache_q4(key[:0], val[:0], kc, vc, slots[:0])  # no tokens
    assert pa.gather_cache_q4(kc, vc, slots[:0])[0].shape == (0, hkv, 256)
    assert pa.device_errors() == 0


def _case(pa, lens, bs, hq, hkv, seed=0, rows=None, scale_k=1.0, scale_v=1.0, spare=2, max_blocks=None):
    """Sequences in a shuffled pool whose unused places hold all ones (steps of NaN)."""
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
    kc = torch.full(pa.q4_cache_shape(pool, bs, hkv), 0xFF, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    pa.reshape_and_cache_q4(k.to(torch.bfloat16), v.to(torch.bfloat16), kc, vc, slots)
    q = torch.randn(len(lens) if rows is None else rows, hq, 256, generator=g, device="cuda").to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, table=table, bt=torch.from_numpy(table).cuda(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), bs=bs, slots=slots)


def _decode(pa, c, scale=0.0625, max_len=None, **kw):
    return pa.decode_q4(c["q"], c["kc"], c["vc"], c["bt"], c["lens"], scale,
                        max_len or max(1, int(c["lens"].max())), **kw)


def _check_decode(out, c, scale=0.0625):
    ref, tol = _q4.decode(_q4.f64(c["q"]), c["kc"].cpu().numpy(), c["vc"].cpu().numpy(), c["bs"],
                          c["table"], c["lens"].cpu().numpy(), scale)
    d = np.abs(_q4.f64(out) - ref)
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


# Shares long enough that a pair's beginning counts (16 tiles and more a CTA): many pairs a CTA,
# empty and one-token sequences between them, and a few pairs that many CTAs share.
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


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_decode_scales(cuda_lib, scale):
    c = _case(cuda_lib, [300, 17], 64, 6, 1, seed=9)
    _check_decode(_decode(cuda_lib, c, scale), c, scale)


@pytest.mark.parametrize("q,k,v", [(1e-3, 1e3, 1e-20), (1e4, 1e-4, 1e20), (1e30, 1e-30, 1.0),
                                   (1e-30, 1.0, 3e4)])
def test_decode_magnitudes(cuda_lib, q, k, v):
    c = _case(cuda_lib, [700], 64, 6, 1, seed=4, scale_k=k, scale_v=v)
    c["q"] = c["q"] * q
    _check_decode(_decode(cuda_lib, c), c)


def test_decode_groups_of_very_different_steps(cuda_lib):
    # One group of V 2^24 times as large as another: each keeps the precision of its own.
    pa = cuda_lib
    c = _case(pa, [500], 64, 4, 1, seed=11)
    N = c["slots"].numel()
    v = torch.randn(N, 1, 4, 64, device="cuda") * torch.tensor([2.0**20, 1.0, 2.0**-4, 8.0], device="cuda")[:, None]
    k = torch.randn(N, 1, 256, device="cuda").to(torch.bfloat16)
    pa.reshape_and_cache_q4(k, v.flatten(-2).to(torch.bfloat16), c["kc"], c["vc"], c["slots"])
    _check_decode(_decode(pa, c), c)


def test_decode_zero_steps_and_zero_query(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [130], 64, 4, 1, seed=12)
    k = torch.randn(130, 1, 1, device="cuda").expand(130, 1, 256).to(torch.bfloat16).contiguous()
    pa.reshape_and_cache_q4(k, k, c["kc"], c["vc"], c["slots"])  # every group constant
    _check_decode(_decode(pa, c), c)
    c["q"].zero_()
    _check_decode(_decode(pa, c), c)


def test_decode_nan_token_reaches_only_its_group_or_heads(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [100], 64, 8, 2, seed=13)
    x = torch.randn(1, 2, 256, device="cuda").to(torch.bfloat16)
    y = x.clone()
    y[0, 1, 70] = float("nan")
    pa.reshape_and_cache_q4(x, y, c["kc"], c["vc"], c["slots"][50:51])  # V of head 1, group 1
    out = _decode(pa, c)
    nan = torch.isnan(out[0])
    assert nan[4:, 64:128].all() and not nan[:4].any() and not nan[4:, :64].any() and not nan[4:, 128:].any()


def test_decode_bad_pages_and_lengths_are_reported(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [70, 200], 64, 6, 1, seed=14)
    c["bt"][1, 1] = 10 ** 6
    out = _decode(pa, c)
    assert pa.device_errors() == pa.DEVERR_PAGE
    cache = c["kc"].cpu().numpy(), c["vc"].cpu().numpy()
    # the page's 64 tokens read as zeros: score 0, value 0
    q = _q4.f64(c["q"])[1]
    kk, vv = (_q4.keys(x, 64, np.where(c["table"][1] < 0, 0, c["table"][1]), 200, 0)[0] for x in cache)
    kk[64:128] = vv[64:128] = 0
    ref = _q4.attend(q, kk, vv, 0.0625, [200] * 6)
    assert np.abs(_q4.f64(out[1]) - ref).max() <= 2e-2
    c["lens"][0] = -3
    c["lens"][1] = 10 ** 6
    c["bt"].clamp_(0, 3)
    out = _decode(pa, c, max_len=200)
    assert pa.device_errors() == pa.DEVERR_SEQLEN
    assert not out[0].any() and torch.isfinite(out[1]).all()


def test_decode_table_wider_than_needed_and_strided(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [100, 333], 64, 6, 1, seed=15, max_blocks=9)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :9] = c["bt"]
    a = _decode(pa, c, max_len=9 * 64)
    c["bt"] = wide[:, :9]
    b = _decode(pa, c, max_len=9 * 64)
    _check_decode(a, c)
    assert torch.equal(a, b)


def test_decode_deterministic_dirty_workspace_and_stream(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [3000, 1, 900], 64, 24, 4, seed=16)
    need = pa.decode_q4_workspace_size(3, 24, 4, 256, 64, 3000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    a = _decode(pa, c, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _decode(pa, c, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    assert torch.equal(a, b)
    _check_decode(a, c)
    with pytest.raises(pa.PAError):
        _decode(pa, c, workspace=ws[:need - 1])


def test_decode_two_graphs_with_their_own_workspaces(cuda_lib):
    pa = cuda_lib
    cs = [_case(pa, [1000 + 77 * i, 5], 64, 24, 4, seed=20 + i, max_blocks=18) for i in range(2)]
    outs, graphs = [], []
    for c in cs:
        ws = torch.empty(pa.decode_q4_workspace_size(2, 24, 4, 256, 64, 1100), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c["q"])
        _decode(pa, c, max_len=1100, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _decode(pa, c, max_len=1100, out=out, workspace=ws)
        outs.append(out)
        graphs.append((g, ws))
    for c in cs:  # other inputs in the same tensors, replayed interleaved
        c["q"].copy_(torch.randn_like(c["q"]))
    for g, _ in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        _check_decode(o, c)


def test_decode_offsets_past_32_bits(cuda_lib):
    # A pool of 4.5 GB per cache: the sequence lies in its last pages.
    pa = cuda_lib
    bs, hkv, pages = 832, 4, 9400
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    kc = torch.empty(pa.q4_cache_shape(pages, bs, hkv), dtype=torch.uint8, device="cuda")
    vc = torch.empty_like(kc)
    assert kc.numel() > 1 << 32
    n = 1000
    slots = torch.cat([(pages - 1) * bs + torch.arange(bs), (pages - 2) * bs + torch.arange(n - bs)]).cuda()
    k, v = (torch.randn(n, hkv, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    pa.reshape_and_cache_q4(k, v, kc, vc, slots)
    table = np.array([[pages - 1, pages - 2]], np.int32)
    q = torch.randn(1, 24, 256, device="cuda").to(torch.bfloat16)
    out = pa.decode_q4(q, kc, vc, torch.from_numpy(table).cuda(),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), 0.0625, n)
    small = dict(q=q, kc=kc[-2:], vc=vc[-2:], bs=bs, table=np.array([[1, 0]], np.int32),
                 lens=torch.tensor([n], dtype=torch.int32))
    _check_decode(out, small)


# ------------------------------------------------------------------------------ prefill
def _check_prefill(got, c, cu, lens, causal=True, scale=0.0625):
    """Each output within the bound, and all of them together within a BF16 rounding's norm
    (at most 2^-8 / sqrt(3) of theirs, errors spread evenly over half a step) and a fifth."""
    ref, tol = _q4.prefill(_q4.f64(c["q"]), c["kc"].cpu().numpy(), c["vc"].cpu().numpy(), c["bs"],
                           c["table"], cu, lens, causal, scale)
    d = np.abs(_q4.f64(got) - ref)
    assert np.isfinite(d).all()
    assert (d <= tol).all(), (d.max(), (d / tol).max())
    assert np.linalg.norm(d) <= np.linalg.norm(ref) * 2.0 ** -8 / 3 ** 0.5 * 1.2


@pytest.mark.parametrize("q_len,q_start,bs,hq,hkv,causal", [
    (1, 0, 64, 6, 1, True), (1, 700, 64, 6, 1, True), (130, 900, 832, 24, 4, True),
    (128, 0, 16, 8, 8, True), (257, 63, 100, 4, 2, True), (40, 300, 784, 6, 1, False),
    (21, 1500, 16, 16, 2, True), (300, 0, 7, 5, 1, True),
])
def test_prefill_chunk_matches_plain(cuda_lib, q_len, q_start, bs, hq, hkv, causal):
    pa = cuda_lib
    n = q_len + q_start
    c = _case(pa, [n], bs, hq, hkv, seed=q_len + bs, rows=q_len)
    out = pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], q_start, causal, 0.0625)
    _check_prefill(out, c, [0, q_len], [n], causal)
    assert pa.device_errors() == 0


def test_prefill_varlen_over_two_launches_and_empty_chunks(cuda_lib):
    pa = cuda_lib
    rng = np.random.default_rng(3)
    rows = [int(x) for x in rng.integers(0, 40, 40)]
    rows[5] = rows[17] = 0
    lens = [r + int(x) for r, x in zip(rows, rng.integers(1, 300, 40))]
    cu = [0] + np.cumsum(rows).tolist()
    c = _case(pa, lens, 16, 12, 4, seed=31, rows=cu[-1])
    need = pa.prefill_varlen_q4_workspace_size(cu, lens, True, 12, 4, 256, 16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = pa.prefill_varlen_q4(c["q"], c["kc"], c["vc"], c["bt"], cu, lens, True, 0.0625, workspace=ws)
    _check_prefill(out, c, cu, lens)
    assert torch.equal(out, pa.prefill_varlen_q4(c["q"], c["kc"], c["vc"], c["bt"], cu, lens, True,
                                                 0.0625))
    assert pa.device_errors() == 0


def test_prefill_split_items_and_less_workspace(cuda_lib):
    # A short chunk over a long context: its items are split along the keys when there is
    # room, and run whole when there is not.
    pa = cuda_lib
    c = _case(pa, [9000], 832, 24, 4, seed=33, rows=60)
    need = pa.prefill_q4_workspace_size(60, 8940, True, 24, 4, 256, 832)
    outs = []
    fixed = need
    for cut in (0, 1):
        ws = torch.empty(fixed - cut, dtype=torch.uint8, device="cuda")
        outs.append(pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], 8940, True, 0.0625, workspace=ws))
        _check_prefill(outs[-1], c, [0, 60], [9000])
    with pytest.raises(pa.PAError):
        pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], 8940, True, 0.0625,
                            workspace=torch.empty(9000 * 4 * 1024, dtype=torch.uint8, device="cuda"))
    assert pa.device_errors() == 0


def test_prefill_many_short_items_a_cta(cuda_lib):
    # Several items a CTA, of one, two and three 128-key halves each, so that items begin on
    # either parity; chunk lengths at and around a query tile's rows.
    pa = cuda_lib
    rows = [1, 127, 128, 129, 130, 2, 64, 200, 16, 17, 96, 128] * 2
    lens = [r + 61 * (i % 5) for i, r in enumerate(rows)]
    cu = [0] + np.cumsum(rows).tolist()
    c = _case(pa, lens, 16, 32, 8, seed=50, rows=cu[-1])
    out = pa.prefill_varlen_q4(c["q"], c["kc"], c["vc"], c["bt"], cu, lens, True, 0.0625)
    _check_prefill(out, c, cu, lens)
    assert torch.equal(out, pa.prefill_varlen_q4(c["q"], c["kc"], c["vc"], c["bt"], cu, lens, True, 0.0625))
    assert pa.device_errors() == 0


@pytest.mark.parametrize("scale", [0.0, -0.0625, 0.0625])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_scores_that_grow_along_the_keys(cuda_lib, scale, causal):
    # Keys up to 16 times as long at the end as at the start: the row's reference moves again
    # and again, in both directions of the scores, and rows end in any half.
    pa = cuda_lib
    n, rows = 1500, 400
    c = _case(pa, [n], 64, 8, 2, seed=51, rows=rows)
    k = torch.randn(n, 2, 256, device="cuda") * torch.linspace(1, 16, n, device="cuda")[:, None, None]
    v = torch.randn(n, 2, 256, device="cuda") + 3
    pa.reshape_and_cache_q4(k.to(torch.bfloat16), v.to(torch.bfloat16), c["kc"], c["vc"], c["slots"])
    out = pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], n - rows, causal, scale)
    ref, tol = _q4.prefill(_q4.f64(c["q"]), c["kc"].cpu().numpy(), c["vc"].cpu().numpy(), 64,
                           c["table"], [0, rows], [n], causal, scale)
    assert (np.abs(_q4.f64(out) - ref) <= tol).all()
    assert pa.device_errors() == 0


@pytest.mark.parametrize("q,k,v", [(1e-3, 1e3, 1e-20), (1e4, 1e-4, 1e20), (1e20, 1e-20, 1e-6)])
def test_prefill_magnitudes(cuda_lib, q, k, v):
    pa = cuda_lib
    c = _case(pa, [200], 64, 6, 1, seed=35, rows=100, scale_k=k, scale_v=v)
    c["q"] = c["q"] * q
    out = pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], 100, True, 0.0625)
    _check_prefill(out, c, [0, 100], [200])


def test_prefill_in_a_graph_beside_another(cuda_lib):
    pa = cuda_lib
    cs = [_case(pa, [400 + i], 64, 12, 2, seed=40 + i, rows=150) for i in range(2)]
    runs = []
    for c in cs:
        n = int(c["lens"][0])
        ws = torch.empty(pa.prefill_q4_workspace_size(150, n - 150, True, 12, 2, 256, 64), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c["q"])
        args = (c["q"], c["kc"], c["vc"], c["bt"][0].contiguous(), n - 150, True, 0.0625, out, ws)
        pa.prefill_chunk_q4(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.prefill_chunk_q4(*args)
        out.zero_()
        runs.append((g, out, args))
    for g, _, _ in runs * 2:
        g.replay()
    torch.cuda.synchronize()
    for c, (_, out, _) in zip(cs, runs):
        n = int(c["lens"][0])
        _check_prefill(out, c, [0, 150], [n])


def test_prefill_bad_page_is_reported(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [200], 64, 6, 1, seed=36, rows=10)
    c["bt"][0, 1] = -1
    out = pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], 190, True, 0.0625)
    assert pa.device_errors() == pa.DEVERR_PAGE
    assert torch.isfinite(out).all()


def test_device_and_layout_refusals(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [20], 16, 6, 1)
    with pytest.raises(ValueError):
        _decode(pa, c, max_len=40)  # the table row is too short
    with pytest.raises(ValueError):
        pa.decode_q4(c["q"], c["kc"], c["vc"][:, :, :144], c["bt"], c["lens"], 0.1, 20)
    with pytest.raises(TypeError):
        pa.decode_q4(c["q"].float(), c["kc"], c["vc"], c["bt"], c["lens"], 0.1, 20)
    with pytest.raises(ValueError):
        pa.decode_q4(c["q"], c["kc"], c["vc"], c["bt"].expand(2, -1)[:0], c["lens"], 0.1, 20)
    with pytest.raises(ValueError):
        pa.reshape_and_cache_q4(c["q"][:, :2], c["q"][:, :2], c["kc"], c["vc"], c["slots"][:1])
