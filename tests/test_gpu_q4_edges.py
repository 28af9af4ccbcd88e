"""Decode over the 4-bit cache at the ends of its range."""
import pytest
import torch

from test_gpu_q4 import _bf, _case, _decode
from test_gpu_q4_accuracy import _check

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ NaN
def test_decode_nan_value_of_vanishing_weight(cuda_lib):
    # The first keys outweigh the rest by e^200: the NaN is in another part, of weight 0 in fp32.
    pa = cuda_lib
    c = _case(pa, [9000], 64, 8, 2, seed=1)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(256, generator=g)
    c["q"] = _bf(q.expand(1, 8, 256))
    x = torch.randn(9000, 2, 256, generator=g)
    x[:8] += (q * (200 / 0.0625 / float(q @ q)))[None, None]
    y = torch.randn(9000, 2, 256, generator=g)
    pa.reshape_and_cache_q4(_bf(x), _bf(y), c["kc"], c["vc"], c["slots"])
    fine = c["vc"].clone()
    for at in range(100, 9000, 300):
        y[at, 1, 70] = float("nan")
        c["vc"].copy_(fine)
        pa.reshape_and_cache_q4(_bf(x[at:at + 1]), _bf(y[at:at + 1]), c["kc"], c["vc"], c["slots"][at:at + 1])
        nan = torch.isnan(_decode(pa, c)[0])
        assert nan[4:, 64:128].all(), at
        assert not nan[:4].any() and not nan[4:, :64].any() and not nan[4:, 128:].any(), at


@pytest.mark.parametrize("n,first,last", [(9000, 4000, 5000), (9000, 0, 9000), (300, 128, 256), (40, 0, 40)])
def test_decode_nan_keys(cuda_lib, n, first, last):
    # Whole shares of NaN keys in head 1: its query heads are NaN, head 0's as they are without.
    pa = cuda_lib
    c = _case(pa, [n], 64, 8, 2, seed=2)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, 2, 256, generator=g) for _ in range(2))
    k[first:last, 1] = float("nan")
    pa.reshape_and_cache_q4(_bf(k), _bf(v), c["kc"], c["vc"], c["slots"])
    out = _decode(pa, c)
    assert torch.isnan(out[0, 4:]).all()
    one = dict(c, q=c["q"][:, :4], kc=c["kc"][:, :1].contiguous(), vc=c["vc"][:, :1].contiguous())
    _check(out[:, :4], one)


# ------------------------------------------------------------------------------ lengths
@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [0] * 40])
@pytest.mark.parametrize("max_len", [1, 100, 9000])
def test_decode_of_padding_entries_alone(cuda_lib, lens, max_len):
    pa = cuda_lib
    c = _case(pa, [64], 64, 8, 2, seed=3)
    S = len(lens)
    q = torch.randn(S, 8, 256, device="cuda").to(torch.bfloat16)
    need = pa.decode_q4_workspace_size(S, 8, 2, 256, 64, max_len)
    for fill in (0, 0xFF):
        out = torch.full_like(q, 3.0)
        pa.decode_q4(q, c["kc"], c["vc"], torch.full((S, 141), -1, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.0625, max_len, out=out,
                     workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        assert not out.any()
    assert pa.device_errors() == 0


def test_decode_lengths_past_the_limit_leave_the_output(cuda_lib):
    # 16 x 2^27 tiles: refused on the device, with the parts of an earlier call in the workspace.
    pa = cuda_lib
    bs, S = 1 << 20, 16
    kc, vc = (torch.zeros(pa.q4_cache_shape(1, bs, 1), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.zeros(S, 2048, dtype=torch.int32, device="cuda")
    q = torch.randn(S, 4, 256, device="cuda").to(torch.bfloat16)
    most = 2**31 - 1
    ws = torch.zeros(pa.decode_q4_workspace_size(S, 4, 1, 256, bs, most), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    lens = torch.full((S,), 5000, dtype=torch.int32, device="cuda")
    pa.decode_q4(q, kc, vc, table, lens, 0.0625, most, out=out, workspace=ws)
    assert pa.device_errors() == 0 and not out.any()
    out.fill_(3.0)
    lens.fill_(most)
    pa.decode_q4(q, kc, vc, table, lens, 0.0625, most, out=out, workspace=ws)
    assert pa.device_errors() == pa.DEVERR_SEQLEN
    assert (out == 3.0).all()


def test_decode_short_sequence_under_the_largest_length(cuda_lib):
    # One sequence of 100 keys whose table has room for 2^31 - 1: no error.
    pa = cuda_lib
    bs, hkv = 1 << 16, 16
    kc, vc = (torch.zeros(pa.q4_cache_shape(1, bs, hkv), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.zeros(1, 1 << 15, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, 256, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(100, hkv, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    pa.reshape_and_cache_q4(k, v, kc, vc, torch.arange(100, device="cuda"))
    lens = torch.tensor([100], dtype=torch.int32, device="cuda")
    out = pa.decode_q4(q, kc, vc, table, lens, 0.0625, 2**31 - 1)
    assert pa.device_errors() == 0
    assert torch.equal(out, pa.decode_q4(q, kc, vc, table, lens, 0.0625, 100))


# ------------------------------------------------------------------------------ steps with idle entries
def _step(pa, new, num_tokens, seed):
    """Prep, norm + rotation and write of one token for each live entry over filled caches."""
    S, bs, pages = len(new), 16, 60
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    computed = [70, 0, 33, 48, 15][:S]
    table = torch.arange(S * 8, device="cuda", dtype=torch.int32).view(S, 8)
    kc, vc = (torch.zeros(pa.q4_cache_shape(pages, bs, 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(S * 8 * bs, device="cuda")
    pa.reshape_and_cache_q4(rn(S * 8 * bs, 2, 256), rn(S * 8 * bs, 2, 256), kc, vc, slots)
    tensor = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    step = pa.batch_input_prep(tensor(computed), tensor(new), [table], [bs],
                               [torch.arange(S * 8, pages, device="cuda", dtype=torch.int32)], num_tokens)
    q, k, v = rn(num_tokens, 8, 256), rn(num_tokens, 2, 256), rn(num_tokens, 2, 256)
    angle = torch.arange(100, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    w = rn(256)
    q = pa.qk_norm_rope_cache(q, k, v, w, w, torch.cat([angle.cos(), angle.sin()], 1), step["positions"], 1e-6,
                              kc, vc, step["slot_mappings"][0])
    return dict(q=q, kc=kc, vc=vc, bt=table, table=table.cpu().numpy(), lens=step["seq_lens"], bs=bs), step


def test_decode_step_with_idle_entries_behind(cuda_lib):
    pa = cuda_lib
    c, _ = _step(pa, [1, 1, 1, 0, 0], 5, 1)
    out = _decode(pa, c)
    assert not out[3:].any()
    live = dict(c, q=c["q"][:3], table=c["table"][:3], bt=c["bt"][:3], lens=c["lens"][:3])
    _check(out[:3], live)
    assert pa.device_errors() == 0


def test_decode_step_with_an_idle_entry_between(cuda_lib):
    # Row 1 of the packed q belongs to entry 2: refused as it is, right when moved there.
    pa = cuda_lib
    c, step = _step(pa, [1, 0, 1, 1, 0], 3, 2)
    packed = c["q"]
    for rows in (packed, torch.cat([packed] * 2)):
        with pytest.raises(ValueError):
            pa.decode_q4(rows, c["kc"], c["vc"], c["bt"], c["lens"], 0.0625, 100)
    c["q"] = torch.zeros(5, 8, 256, dtype=torch.bfloat16, device="cuda")
    c["q"][step["seq_idx"].long()] = packed
    out = _decode(pa, c)
    _check(out, c)
    assert not out[[1, 4]].any() and pa.device_errors() == 0


def test_lengths_past_32_bits_are_refused(cuda_lib):
    pa = cuda_lib
    c = _case(pa, [20], 1 << 16, 6, 1, seed=9, max_blocks=(1 << 16) + 1)
    with pytest.raises(ValueError):
        _decode(pa, c, max_len=2**32 + 20)
    for q_start in (2**32 + 19, 2**31 - 1):
        with pytest.raises(ValueError):
            pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], q_start, True, 0.0625)
    with pytest.raises(pa.PAError):
        pa.prefill_chunk_q4(c["q"], c["kc"], c["vc"], c["bt"][0], -1, True, 0.0625)


def test_prep_lengths_of_the_step_before(cuda_lib):
    # Many CTAs read the lengths: in place they are refused, a copy is taken.
    pa = cuda_lib
    S, T = 600, 9000
    new = torch.full((S,), 15, dtype=torch.int32, device="cuda")
    table = torch.full((S, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(4 * S, dtype=torch.int32, device="cuda")
    out = pa.batch_input_prep(torch.zeros_like(new), new, [table], [16], [free], T)
    assert out["pages_taken"].tolist() == [S]
    with pytest.raises(pa.PAError):
        pa.batch_input_prep(out["seq_lens"], new, [table], [16], [free[S:]], T, out=out)
    out = pa.batch_input_prep(out["seq_lens"].clone(), new, [table], [16], [free[S:]], T, out=out)
    assert out["seq_lens"].tolist() == [30] * S and out["pages_taken"].tolist() == [S]
    assert out["positions"].view(S, 15)[:, 0].tolist() == [15] * S
    assert torch.equal(table[:, :2], torch.stack([free[:S], free[S:2 * S]], 1))
    assert pa.device_errors() == 0
