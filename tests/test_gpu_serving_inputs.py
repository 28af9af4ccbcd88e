"""Mixed-step inputs, norm + rotation, and whole steps over the 4-bit cache, on the GPU."""
import numpy as np
import pytest
import torch

import _q4

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ batch prep
def _prep_case(S, sizes, T, seed, ctx=3000, idle=5):
    rng = np.random.default_rng(seed)
    computed = rng.integers(0, ctx + 1, S).astype(np.int32)
    new = np.ones(S, np.int32)
    if S:
        share = rng.random(S) * (rng.random(S) < 0.3)
        new += (share / max(share.sum(), 1e-9) * max(T - S, 0) * 0.95).astype(np.int32)
        new[::idle] = rng.integers(-2, 1, new[::idle].shape)
    tables, free = [], []
    for bs in sizes:
        width = -(-(ctx + int(new.max(initial=0))) // bs) + 1
        ids = rng.permutation(4 * (S * width + 10)).astype(np.int32)
        t = np.full((S, width), -1, np.int32)
        at = 0
        for s in range(S):
            m = -(-int(computed[s]) // bs)
            t[s, :m] = ids[at:at + m]
            at += m
        need = int(sum(-(-int(c + n) // bs) - -(-int(c) // bs) for c, n in zip(computed, new) if n > 0))
        tables.append(t)
        free.append(ids[at:at + need + 3])
    return computed, new, tables, free


def _run_prep(pa, computed, new, tables, sizes, free, T, **kw):
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    tt = [cuda(t) for t in tables]
    got = pa.batch_input_prep(cuda(computed), cuda(new), tt, sizes, [cuda(f) for f in free], T, **kw)
    return got, tt


def _same_prep(got, tables, want, T):
    for k in ("seq_lens", "query_start_loc", "positions", "seq_idx", "pages_taken"):
        assert np.array_equal(got[k].cpu().numpy(), want[k]), k
    for a, b in zip(got["slot_mappings"], want["slot_mappings"]):
        assert np.array_equal(a.cpu().numpy(), b)
    for a, b in zip(tables, want["tables"]):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("S,sizes,T", [
    (1, [832], 1), (1, [16], 5000), (16, [832], 16), (33, [16, 832], 3000), (257, [64], 1024),
    (300, [7, 1, 16], 2049), (1000, [784], 4096), (3000, [832, 16], 3100),
    (9, [5, 832, 784, 64, 16, 2, 3, 1], 1500),
])
def test_batch_prep_matches_plain(cuda_lib, S, sizes, T):
    pa = cuda_lib
    computed, new, tables, free = _prep_case(S, sizes, T, S + T)
    want, short = _q4.batch_prep(computed, new, tables, sizes, free, T)
    got, tt = _run_prep(pa, computed, new, tables, sizes, free, T)
    assert not short
    _same_prep(got, tt, want, T)
    assert pa.device_errors() == 0


def test_batch_prep_edges(cuda_lib):
    pa = cuda_lib
    # no sequences; only idle entries; one token at a page border
    got, _ = _run_prep(pa, np.zeros(0, np.int32), np.zeros(0, np.int32), [np.zeros((0, 4), np.int32)], [16],
                       [np.arange(3, dtype=np.int32)], 5)
    assert got["query_start_loc"].tolist() == [0] and got["positions"].tolist() == [-1] * 5
    assert got["pages_taken"].tolist() == [0]
    got, tt = _run_prep(pa, np.array([16, 5], np.int32), np.array([0, -3], np.int32),
                        [np.array([[4, -1], [5, -1]], np.int32)], [16], [np.array([9], np.int32)], 2)
    assert got["seq_lens"].tolist() == [0, 0] and got["slot_mappings"][0].tolist() == [-1, -1]
    assert tt[0].tolist() == [[4, -1], [5, -1]]
    got, tt = _run_prep(pa, np.array([16], np.int32), np.array([1], np.int32),
                        [np.array([[4, -1]], np.int32)], [16], [np.array([9], np.int32)], 1)
    assert tt[0].tolist() == [[4, 9]] and got["slot_mappings"][0].tolist() == [144]
    assert pa.device_errors() == 0


def test_batch_prep_reports_what_it_cannot_do(cuda_lib):
    pa = cuda_lib
    one = lambda *x: np.array(x, np.int32)
    # the free list runs out
    got, tt = _run_prep(pa, one(0, 0), one(20, 20), [np.full((2, 3), -1, np.int32)], [16], [one(7, 8, 9)], 40)
    want, short = _q4.batch_prep(one(0, 0), one(20, 20), [np.full((2, 3), -1, np.int32)], [16], [one(7, 8, 9)], 40)
    assert short and pa.device_errors() == pa.DEVERR_NO_PAGES
    _same_prep(got, tt, want, 40)
    # a logical page past the row: no page is taken for it
    got, tt = _run_prep(pa, one(30, 0), one(10, 1), [np.array([[1, 2], [-1, -1]], np.int32)], [16],
                        [one(7, 8)], 11)
    assert pa.device_errors() == pa.DEVERR_POSITION
    assert got["slot_mappings"][0].tolist() == [46, 47] + [-1] * 8 + [7 * 16]
    assert tt[0].tolist() == [[1, 2], [7, -1]]
    # more tokens than rows
    got, tt = _run_prep(pa, one(0, 0), one(6, 6), [np.full((2, 2), -1, np.int32)], [4], [one(3, 4, 5, 6)], 9)
    assert pa.device_errors() == pa.DEVERR_POSITION
    assert got["query_start_loc"].tolist() == [0, 6, 12] and got["seq_idx"].tolist() == [0] * 6 + [1] * 3
    assert tt[0].tolist() == [[3, 4], [5, -1]]
    # a negative entry of a page held before, and of the free list
    got, _ = _run_prep(pa, one(3, 0), one(1, 1), [np.array([[-1], [-1]], np.int32)], [16], [one(-4)], 2)
    assert pa.device_errors() == pa.DEVERR_POSITION and got["slot_mappings"][0].tolist() == [-1, -1]
    # impossible lengths are idle
    got, _ = _run_prep(pa, one(-1, 2**31 - 5, 0), one(2, 10, 1), [np.full((3, 1), 2, np.int32)], [16],
                       [one(6)], 3)
    assert pa.device_errors() == pa.DEVERR_SEQLEN
    assert got["seq_lens"].tolist() == [0, 0, 1] and got["positions"].tolist() == [0, -1, -1]


def test_batch_prep_agrees_with_decode_input_prep(cuda_lib):
    # A decode step is the special case of one new token per sequence.
    pa = cuda_lib
    rng = np.random.default_rng(2)
    S = 200
    computed = rng.integers(0, 5000, S).astype(np.int32)
    tables = [rng.permutation(S * n).astype(np.int32).reshape(S, n) for n in (7, 320)]
    cuda = lambda a: torch.from_numpy(a).cuda()
    want = pa.decode_input_prep(cuda(computed), [cuda(t) for t in tables], [832, 16])
    free = [np.array([tables[g][s, computed[s] // bs] for s in range(S) if computed[s] % bs == 0] or [0], np.int32)
            for g, bs in enumerate((832, 16))]
    got, _ = _run_prep(pa, computed, np.ones(S, np.int32), tables, [832, 16], free, S)
    assert torch.equal(got["seq_lens"], want["seq_lens"])
    assert torch.equal(got["query_start_loc"], want["query_start_loc"])
    for a, b in zip(got["slot_mappings"], want["slot_mappings"]):
        assert torch.equal(a, b)


def test_batch_prep_graph_and_reused_outputs(cuda_lib):
    pa = cuda_lib
    computed, new, tables, free = _prep_case(50, [16, 64], 700, 5)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    c, n, tt, ff = cuda(computed), cuda(new), [cuda(t) for t in tables], [cuda(f) for f in free]
    out = pa.batch_input_prep(c, n, [t.clone() for t in tt], [16, 64], ff, 700)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.batch_input_prep(c, n, tt, [16, 64], ff, 700, out=out)
    n.copy_(torch.flip(n, [0]))  # other lengths in the captured tensors
    g.replay()
    torch.cuda.synchronize()
    want, _ = _q4.batch_prep(computed, new[::-1], tables, [16, 64], free, 700)
    _same_prep(out, tt, want, 700)
    pa.device_errors()
    with pytest.raises(ValueError):
        pa.batch_input_prep(c, n, tt, [16, 64], ff, 701, out=out)


# ------------------------------------------------------------------------------ norm + rotation
def _rope_case(T, hq, hkv, dim, rot, rows=500, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randn(T, (hq + 2 * hkv) * dim, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in packed.split([hq * dim, hkv * dim, hkv * dim], 1))
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, rows, (T,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.from_numpy(_q4.cos_sin_table(rows, rot)).cuda()
    return q, k, v, w, table, pos


def _rope_ref(x, w, table, pos, interleaved, bias=0.0, eps=1e-6):
    """fp64 rows and the bound: half a BF16 step of the result, and fp32's share of the pair that
    it is made of (a dozen roundings of 2^-24 on values of the row's size)."""
    y = _q4.rope(_q4.f64(x), _q4.f64(w), bias, eps, table.double().cpu().numpy(), pos.tolist(), interleaved)
    plain = _q4.rope(_q4.f64(x), _q4.f64(w), bias, eps, np.zeros((1, 0)), [-1] * len(y), interleaved)
    big = np.abs(plain).max(-1, keepdims=True)
    return y, np.abs(y) * 2.0 ** -8 * 1.01 + 2.0 ** -19 * big + 1e-30


@pytest.mark.parametrize("dim,rot,hq,hkv,T,interleaved", [
    (256, 64, 24, 4, 16, False), (256, 256, 24, 4, 3, False), (256, 64, 5, 1, 1, True),
    (128, 128, 32, 8, 40, False), (128, 32, 6, 2, 7, True), (64, 64, 9, 3, 20, False),
    (64, 16, 3, 1, 5, True), (256, 0, 8, 2, 4, False), (256, 256, 7, 7, 600, True),
    (128, 16, 1, 1, 513, False),
])
def test_rope_matches_plain(cuda_lib, dim, rot, hq, hkv, T, interleaved):
    pa = cuda_lib
    q, k, v, w, table, pos = _rope_case(T, hq, hkv, dim, rot)
    qo, ko = pa.qk_norm_rope(q, k, w[0], w[1], table, pos, 1e-6, interleaved=interleaved)
    for got, x, ww in ((qo, q, w[0]), (ko, k, w[1])):
        ref, tol = _rope_ref(x, ww, table, pos, interleaved)
        assert (np.abs(_q4.f64(got) - ref) <= tol).all()
    assert pa.device_errors() == 0


def test_rope_weight_bias_zero_rows_and_eps(cuda_lib):
    pa = cuda_lib
    q, k, v, w, table, pos = _rope_case(6, 4, 2, 256, 64)
    q = q.clone()
    q[2] = 0
    small = [x - 1 for x in w]
    qo, ko = pa.qk_norm_rope(q, k, small[0], small[1], table, pos, 0.5, weight_bias=1.0)
    ref, tol = _rope_ref(q, small[0], table, pos, False, 1.0, 0.5)
    assert (np.abs(_q4.f64(qo) - ref) <= tol).all() and not qo[2].any()


def test_rope_in_place_and_padding_rows_left(cuda_lib):
    pa = cuda_lib
    q, k, v, w, table, pos = _rope_case(700, 24, 4, 256, 64, seed=3)
    pos[5] = -1
    pos[699] = 500  # past the table
    want_q, want_k = q.clone(), k.clone()
    qo, ko = pa.qk_norm_rope(q, k, w[0], w[1], table, pos, 1e-6, q_out=want_q, k_out=want_k)
    assert pa.device_errors() == pa.DEVERR_POSITION
    assert torch.equal(want_q[[5, 699]], q[[5, 699]]) and torch.equal(want_k[[5, 699]], k[[5, 699]])
    keep = v.clone()
    pa.qk_norm_rope(q, k, w[0], w[1], table, pos, 1e-6, q_out=q, k_out=k)  # views of one tensor
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(v, keep)
    assert pa.device_errors() == pa.DEVERR_POSITION


@pytest.mark.parametrize("T,dim,bs,interleaved", [(1, 256, 16, False), (16, 256, 832, False), (600, 256, 64, True),
                                                  (9, 128, 16, False), (30, 64, 7, True)])
def test_rope_cache_is_the_two_calls(cuda_lib, T, dim, bs, interleaved):
    pa = cuda_lib
    hq, hkv = 12, 4
    q, k, v, w, table, pos = _rope_case(T, hq, hkv, dim, 64, seed=T)
    if T > 4:
        pos[3] = -1
    qo, ko = pa.qk_norm_rope(q, k, w[0], w[1], table, pos, 1e-6, interleaved=interleaved)
    pages = -(-T // bs) + 1
    slots = torch.randperm(pages * bs, device="cuda")[:T]
    slots[T // 2] = -1
    live = slots.clone()
    if T > 4:
        live[3] = -1
    kv = torch.zeros(pages, 2, bs, hkv, dim, dtype=torch.bfloat16, device="cuda")
    want = torch.zeros_like(kv)
    pa.reshape_and_cache(ko, v, want[:, 0], want[:, 1], live)
    got_q = pa.qk_norm_rope_cache(q, k, v, w[0], w[1], table, pos, 1e-6, kv[:, 0], kv[:, 1], slots,
                                  interleaved=interleaved)
    rows = pos >= 0
    assert torch.equal(got_q[rows], qo[rows]) and torch.equal(kv, want)
    if dim == 256:
        kc = torch.zeros(pa.q4_cache_shape(pages, bs, hkv), dtype=torch.uint8, device="cuda")
        vc, wk, wv = kc.clone(), kc.clone(), kc.clone()
        pa.reshape_and_cache_q4(ko, v, wk, wv, live)
        got_q = pa.qk_norm_rope_cache(q, k, v, w[0], w[1], table, pos, 1e-6, kc, vc, slots,
                                      interleaved=interleaved)
        assert torch.equal(got_q[rows], qo[rows]) and torch.equal(kc, wk) and torch.equal(vc, wv)
    assert pa.device_errors() == 0
    slots[0] = pages * bs
    pa.qk_norm_rope_cache(q, k, v, w[0], w[1], table, pos, 1e-6, kv[:, 0], kv[:, 1], slots)
    assert pa.device_errors() == pa.DEVERR_SLOT


def test_rope_refuses_bad_layouts(cuda_lib):
    pa = cuda_lib
    q, k, v, w, table, pos = _rope_case(4, 4, 2, 256, 64)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, w[0], w[1], table, pos, 1e-6)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(q, k[:3], w[0], w[1], table, pos, 1e-6)
    with pytest.raises(TypeError):
        pa.qk_norm_rope(q, k, w[0].float(), w[1], table, pos, 1e-6)
    with pytest.raises(pa.PAError):
        pa.qk_norm_rope(q, k, w[0], w[1], table[:, :40].contiguous(), pos, 1e-6)


# ------------------------------------------------------------------------------ whole steps
@pytest.mark.parametrize("bs", [16, 784])
def test_serving_steps_over_the_q4_cache(cuda_lib, bs):
    """Three requests: a mixed step (two prompt chunks and a decode), then decode steps, each
    through prep, norm + rotation + write, and attention; against fp64 over the cache."""
    pa = cuda_lib
    hq, hkv, S, pool = 12, 2, 4, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [(1 + 0.1 * torch.randn(256, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    table = torch.from_numpy(_q4.cos_sin_table(4000, 64)).cuda()
    kc = torch.full(pa.q4_cache_shape(pool, bs, hkv), 0xFF, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    free = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((S, -(-2000 // bs)), -1, dtype=torch.int32, device="cuda")
    computed = torch.zeros(S, dtype=torch.int32, device="cuda")
    used = 0
    for step, new in enumerate(([850, 33, 0, 1], [300, 1, 0, 1], [1, 1, 5, 1], [1, 1, 1, 1])):
        T = sum(new)
        prep = pa.batch_input_prep(computed, torch.tensor(new, dtype=torch.int32, device="cuda"), [bt], [bs],
                                   [free[used:]], T)
        used += int(prep["pages_taken"][0])
        packed = torch.randn(T, (hq + 2 * hkv) * 256, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, 256)) for x in packed.split([hq * 256, hkv * 256, hkv * 256], 1))
        qn = pa.qk_norm_rope_cache(q, k, v, w[0], w[1], table, prep["positions"], 1e-6, kc, vc,
                                   prep["slot_mappings"][0])
        cu, lens = prep["query_start_loc"].tolist(), prep["seq_lens"].tolist()
        if max(new) > 1:
            out = pa.prefill_varlen_q4(qn, kc, vc, bt, cu, lens, True, 0.0625)
        else:
            out = pa.decode_q4(qn, kc, vc, bt, prep["seq_lens"], 0.0625, 1400)
        hk, hv, tab = kc.cpu().numpy(), vc.cpu().numpy(), bt.cpu().numpy()
        assert lens == [int(c) + n if n else 0 for c, n in zip(computed, new)]
        args = _q4.f64(qn), hk, hv, bs, tab
        if max(new) > 1:
            ref, tol = _q4.prefill(*args, cu, lens, True, 0.0625)
        else:
            ref, tol = _q4.decode(*args, lens, 0.0625)
        assert (np.abs(_q4.f64(out) - ref) <= tol).all(), step
        # the newest key of sequence 0 is what the norm and rotation say, within a step
        row = cu[1] - 1
        want, _ = _rope_ref(k[row:row + 1], w[1], table, prep["positions"][row:row + 1], False)
        n, s_, lo = _q4.quantise(want)
        last = _q4.keys(hk, bs, tab[0], lens[0], 0)[0][-1]
        assert np.abs(last - want[0, 0]).max() <= s_[0, 0].max() * 0.51 + np.abs(want).max() * 2.0 ** -8
        computed += torch.tensor(new, dtype=torch.int32, device="cuda")
    assert pa.device_errors() == 0
