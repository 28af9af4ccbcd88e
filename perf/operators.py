"""Cases and plain forms of the serving operators around the 4-bit KV cache.

Five operators, as one serving step uses them:

* ``prep``    batch_input_prep: pages, block tables, positions and slots of a mixed batch
              from the requests' lengths;
* ``rope``    qk_norm_rope_cache: RMS norm of each query and key head, rotation by
              position and the KV write, from the packed projection;
* ``write``   reshape_and_cache_q4, then gather_cache_q4: new tokens quantised into the
              4-bit cache, and read back;
* ``decode``  decode_q4: one query token per sequence over the 4-bit cache;
* ``prefill`` prefill_varlen_q4: chunks of query rows over the 4-bit cache.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits.

The 4-bit cache.  A token's row of one head (256 values) is cut into 4 groups of 64.
Group g keeps its minimum lo and a step s = bf16((max - lo) / 15), both BF16, and 64 codes
n = clamp(rint((x - lo) / s), 0, 15) (0 where s is 0); it stands for lo + s * n.  A cache
is uint8 [pages, kv heads, block_size * 144]: for each page and head first the codes,
128 bytes a token, then the (s, lo) pairs, 16 bytes a token.  In a token's 128 bytes unit
u of 16 bytes holds the dims 8u .. 8u+7 of each group, group by group, two codes a byte,
the lower dim in the lower half; it is stored at place u ^ (token's offset in the page % 8).
"""
import math

import torch

own = False

D = 256
GROUPS = 4
ROW_BYTES = 144  # 128 of codes, 4 pairs of BF16
EPS = 1e-6


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # The admission of one decode step of a small server: 16 running requests.
        {"name": "prep 16 requests", "op": "prep", "seqs": 16, "tokens": 16, "ctx": 32768,
         "bs0": 832, "bs1": 0},
        # A mixed step at full load: 512 requests, most of them decoding, the others with
        # prompt chunks, a model of two cache groups.
        {"name": "prep 512 requests 32768 tokens", "op": "prep", "seqs": 512, "tokens": 32768,
         "ctx": 32768, "bs0": 832, "bs1": 16},
        # One layer's query/key step of a decode batch of 16, quarter rotation.
        {"name": "rope 16 tokens", "op": "rope", "tokens": 16, "hq": 24, "hkv": 4, "dim": 256,
         "rotary": 64, "pairs": "halves", "bs": 832, "table": 32768},
        # The same step of a q=4096 prompt chunk, the whole head rotated.
        {"name": "rope 4096 tokens", "op": "rope", "tokens": 4096, "hq": 24, "hkv": 4, "dim": 256,
         "rotary": 256, "pairs": "halves", "bs": 832, "table": 16384},
        # The new tokens of a decode batch of 16.
        {"name": "write 16 tokens", "op": "write", "tokens": 16, "hkv": 4, "bs": 832},
        # The K/V of a q=4096 prompt chunk.
        {"name": "write 4096 tokens", "op": "write", "tokens": 4096, "hkv": 4, "bs": 832},
        # A short single request: latency.
        {"name": "decode 1x1701", "op": "decode", "seqs": 1, "low": 1701, "high": 1701, "hq": 24,
         "hkv": 4, "bs": 832},
        # A single request at the longest context.
        {"name": "decode 1x32768", "op": "decode", "seqs": 1, "low": 32768, "high": 32768,
         "hq": 24, "hkv": 4, "bs": 832},
        # A decode batch of long, uneven contexts.
        {"name": "decode 16x4096..32768", "op": "decode", "seqs": 16, "low": 4096, "high": 32768,
         "hq": 24, "hkv": 4, "bs": 832},
        # Many short requests in small pages, another head layout.
        {"name": "decode 64x1..2048 pages of 16", "op": "decode", "seqs": 64, "low": 1,
         "high": 2048, "hq": 32, "hkv": 8, "bs": 16},
        # A prompt's last, shorter chunk over its earlier tokens.
        {"name": "prefill 1685 over 12288", "op": "prefill", "q0": 1685, "k0": 13973, "q1": 0,
         "k1": 0, "q2": 0, "k2": 0, "hq": 24, "hkv": 4, "bs": 832},
        # A mixed batch: a full chunk, a short one and a request of a few rows.
        {"name": "prefill mixed", "op": "prefill", "q0": 4096, "k0": 8192, "q1": 512, "k1": 512,
         "q2": 5, "k2": 2999, "hq": 24, "hkv": 4, "bs": 784},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["prep", "rope", "write", "decode", "decode", "prefill"])
    hq, hkv = rng.choice([(24, 4), (24, 4), (32, 8), (16, 2), (8, 8), (5, 1), (12, 4)])
    bs = rng.choice([16, 64, 784, 832])
    if op == "prep":
        seqs = _log(rng, 1, 512)
        return {"op": op, "seqs": seqs, "tokens": max(seqs, _log(rng, 1, 32768)),
                "ctx": _log(rng, 16, 32768), "bs0": bs, "bs1": rng.choice([0, 16, 64, 832])}
    if op == "rope":
        dim = rng.choice([256, 256, 128, 64])
        return {"op": op, "tokens": _log(rng, 1, 4096), "hq": hq, "hkv": hkv,
                "dim": dim, "rotary": rng.choice([r for r in (16, 32, 64, 128, 256) if r <= dim]),
                "pairs": rng.choice(["halves", "neighbours"]), "bs": bs,
                "table": _log(rng, 4096, 262144)}
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 4096), "hkv": min(hkv, 4), "bs": bs}
    if op == "decode":
        seqs = _log(rng, 1, 64)
        high = _log(rng, 1, min(32768, 262144 // seqs))
        return {"op": op, "seqs": seqs, "low": rng.choice([1, max(1, high // 8), high]),
                "high": high, "hq": hq, "hkv": hkv, "bs": bs}
    case = {"op": op}
    for i in range(3):
        q = _log(rng, 1, 1685) if i == 0 or rng.random() < 0.5 else 0
        case.update({"q%d" % i: q, "k%d" % i: q + (rng.choice([0, _log(rng, 1, 8192)]) if q else 0)})
    return {**case, "hq": hq, "hkv": hkv, "bs": bs}


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _pick(low, high, count, gen):
    return torch.randint(low, high + 1, (count,), generator=gen, device="cuda", dtype=torch.int32)


def _tables(lens, bs, spare, gen):
    """Block tables of sequences of these lengths over one shuffled pool, -1 past each
    sequence's pages, and the pool's pages."""
    need = [-(-n // bs) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    pages = torch.tensor(need, device="cuda")
    col = torch.arange(max(max(need), 1), device="cuda")
    first = torch.cumsum(pages, 0) - pages
    at = (first[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < pages[:, None], perm[at], perm.new_full((), -1)), pool


def _quantised(x):
    """BF16 rows [.., 256] -> (codes [.., 256] as uint8, steps and minima [.., 4] BF16)."""
    g = x.double().unflatten(-1, (GROUPS, 64))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo).float() / 15.0).to(torch.bfloat16)
    step = s.double().unsqueeze(-1)
    n = torch.where(step > 0, torch.round((g - lo.unsqueeze(-1)) / step.clamp(min=1e-300)), 0.0)
    return n.clamp(0, 15).to(torch.uint8).flatten(-2), s, lo.to(torch.bfloat16)


def _rows(codes, offsets):
    """Codes [.., T, 256] -> the 128 bytes of each token, whose offsets in its page are
    offsets [T]."""
    w = codes.unflatten(-1, (GROUPS, 8, 8)).transpose(-3, -2)  # [.., T, unit, group, 8 dims]
    b = (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-2)        # [.., T, unit, 16 bytes]
    place = torch.arange(8, device=codes.device) ^ (offsets % 8)[:, None]
    return torch.gather(b, -2, place[..., None].expand(b.shape)).flatten(-2)


def _filled_cache(pool, hkv, bs, gen, peaked):
    """A whole pool of 4-bit pages of N(0, 1) rows; 5% of a key cache's rows eight times
    as large."""
    cache = torch.empty((pool, hkv, bs * ROW_BYTES), dtype=torch.uint8, device="cuda")
    at = torch.arange(bs, device="cuda")
    step = max(1, (1 << 25) // (hkv * bs * D))
    for p in range(0, pool, step):
        x = torch.randn((min(step, pool - p), hkv, bs, D), generator=gen, device="cuda")
        if peaked:
            x *= 1 + 7 * (torch.rand(x.shape[:3], generator=gen, device="cuda") < 0.05)[..., None]
        codes, s, lo = _quantised(x.to(torch.bfloat16))
        part = cache[p:p + step]
        part[..., :bs * 128] = _rows(codes, at).flatten(-2)
        part[..., bs * 128:] = torch.stack([s, lo], -1).flatten(-3).view(torch.uint8)
    return cache


def _spoil_tails(cache, table, lens, bs):
    """The last pages' places past each sequence's end hold all ones (steps of NaN)."""
    for s, n in enumerate(lens):
        r = n % bs
        if r:
            page = cache[int(table[s, n // bs])]
            page[:, r * 128:bs * 128] = 255
            page[:, bs * 128 + r * 16:] = 255


def _chunks(case):
    return [(case["q%d" % i], case["k%d" % i]) for i in range(3) if case["k%d" % i]]


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "prep":
        S, T = case["seqs"], case["tokens"]
        # Every fourth request brings a share of the prompt tokens, the others one token.
        share = torch.rand(S, generator=gen, device="cuda")
        share = share * (torch.arange(S, device="cuda") % 4 == 0)
        new = 1 + (share / share.sum().clamp(min=1e-9) * (T - S) * 0.99).to(torch.int32)
        new[_pick(0, S - 1, max(1, S // 16), gen).long()] = 0 if S > 1 else 1  # idle entries
        computed = _pick(0, case["ctx"], S, gen)
        tables, free, sizes = [], [], [b for b in (case["bs0"], case["bs1"]) if b]
        for b in sizes:
            width = -(-(case["ctx"] + T) // b)
            held = S * (-(-case["ctx"] // b))
            perm = torch.randperm(held + S + T // b + 1, generator=gen, device="cuda").to(torch.int32)
            col = torch.arange(width, device="cuda")
            mine = col < ((computed + b - 1) // b)[:, None]
            at = torch.arange(S, device="cuda")[:, None] * (-(-case["ctx"] // b)) + col
            tables.append(torch.where(mine, perm[at.clamp(max=perm.numel() - 1)], perm.new_full((), -1)))
            free.append(perm[held:].contiguous())
        return {"op": op, "computed": computed, "new": new, "tables": tables, "sizes": sizes,
                "free": free, "tokens": T}
    if op == "rope":
        T, hq, hkv, dim, bs = (case[k] for k in ("tokens", "hq", "hkv", "dim", "bs"))
        packed = _normal((T, (hq + 2 * hkv) * dim), gen)  # the projection's output
        q, k, v = (x.unflatten(1, (-1, dim)) for x in packed.split([hq * dim, hkv * dim, hkv * dim], 1))
        rot = case["rotary"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * freq
        pool = -(-T // bs) + 2
        weight = [(1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).to(torch.bfloat16)
                  for _ in range(2)]
        first = int(torch.randint(0, max(1, case["table"] - T), (1,), generator=gen, device="cuda"))
        positions = (first + torch.arange(T, device="cuda")).clamp(max=case["table"] - 1)
        slots = torch.randperm(pool, generator=gen, device="cuda")[torch.arange(T, device="cuda") // bs]
        return {"op": op, "q": q, "k": k, "v": v, "q_weight": weight[0], "k_weight": weight[1],
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
                "neighbours": case["pairs"] == "neighbours", "positions": positions.to(torch.int32),
                "slots": slots * bs + torch.arange(T, device="cuda") % bs,
                "k_cache": _normal((pool, bs, hkv, dim), gen),
                "v_cache": _normal((pool, bs, hkv, dim), gen)}
    if op == "write":
        T, hkv, bs = case["tokens"], case["hkv"], case["bs"]
        pool = -(-T // bs) + 2
        page = torch.randperm(pool, generator=gen, device="cuda")[torch.arange(T, device="cuda") // bs]
        return {"op": op, "key": _normal((T, hkv, D), gen), "value": _normal((T, hkv, D), gen),
                "slots": page * bs + torch.arange(T, device="cuda") % bs, "bs": bs,
                "k_cache": _filled_cache(pool, hkv, bs, gen, True),
                "v_cache": _filled_cache(pool, hkv, bs, gen, False)}
    hq, hkv, bs = case["hq"], case["hkv"], case["bs"]
    if op == "decode":
        lens = _pick(case["low"], case["high"], case["seqs"], gen)
        lens[0] = case["high"]
        lens = lens.tolist()
    else:
        lens = [k for _, k in _chunks(case)]
    table, pool = _tables(lens, bs, 3, gen)
    state = {"op": op, "table": table, "bs": bs, "scale": 1.0 / math.sqrt(D),
             "k_cache": _filled_cache(pool, hkv, bs, gen, True),
             "v_cache": _filled_cache(pool, hkv, bs, gen, False)}
    _spoil_tails(state["k_cache"], table, lens, bs)
    _spoil_tails(state["v_cache"], table, lens, bs)
    if op == "decode":
        return {**state, "q": _normal((len(lens), hq, D), gen), "longest": max(lens),
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    starts = [0]
    for q, _ in _chunks(case):
        starts.append(starts[-1] + q)
    return {**state, "q": _normal((starts[-1], hq, D), gen), "starts": starts, "lens": lens}


# ------------------------------------------------------------------------------ plain forms
def _values(cache, bs):
    """Pages [.., kv heads, block_size * 144] -> the values they stand for, fp32
    [.., kv heads, block_size, 256]."""
    rows = cache[..., :bs * 128].unflatten(-1, (bs, 8, 16))
    place = torch.arange(8, device=cache.device) ^ (torch.arange(bs, device=cache.device) % 8)[:, None]
    rows = torch.gather(rows, -2, place[..., None].expand(rows.shape)).unflatten(-1, (GROUPS, 4))
    codes = torch.stack([rows & 15, rows >> 4], -1).flatten(-2)           # [.., bs, unit, group, 8]
    codes = codes.transpose(-3, -2).flatten(-2)                           # [.., bs, group, 64]
    pairs = cache[..., bs * 128:].contiguous().view(torch.bfloat16).unflatten(-1, (bs, GROUPS, 2)).float()
    return (pairs[..., 1:] + pairs[..., :1] * codes.float()).flatten(-2)


def _sequences(cache, table, bs):
    """Every sequence's values [S, kv heads, pages * block_size, 256]."""
    return _values(cache[table.clamp(min=0).long()], bs).transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, seen, scale):
    """q [.., M, 256] over k, v [.., N, 256]; seen: which keys each row sees.  Rows that
    see none give zeros; what is not seen may hold anything."""
    any_row = seen.any(-2).unsqueeze(-1)
    k, v = k.masked_fill(~any_row, 0), v.masked_fill(~any_row, 0)
    x = (q @ k.transpose(-1, -2) * scale).masked_fill(~seen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    return p @ v / torch.where(total > 0, total, 1.0)


def _plain_decode(st):
    S, hq, _ = st["q"].shape
    hkv = st["k_cache"].shape[1]
    k, v = (_sequences(st[n], st["table"], st["bs"]) for n in ("k_cache", "v_cache"))
    seen = (torch.arange(k.shape[2], device="cuda") < st["lens"][:, None])[:, None, None]
    q = st["q"].float().view(S, hkv, hq // hkv, D)
    return _attend(q, k, v, seen, st["scale"]).view(S, hq, D).to(torch.bfloat16)


def _plain_prefill(st):
    """Every chunk padded to the longest one."""
    total, hq, _ = st["q"].shape
    hkv, dev = st["k_cache"].shape[1], st["q"].device
    k, v = (_sequences(st[n], st["table"], st["bs"]) for n in ("k_cache", "v_cache"))
    starts, lens = torch.tensor(st["starts"], device=dev), torch.tensor(st["lens"], device=dev)
    rows = starts[1:] - starts[:-1]
    i = torch.arange(max(b - a for a, b in zip(st["starts"], st["starts"][1:])), device=dev)
    at = (starts[:-1, None] + i).clamp(max=total - 1)
    q = st["q"][at].float().unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, M, 256]
    last = (lens - rows)[:, None] + i
    seen = torch.arange(k.shape[2], device=dev) <= last.clamp(max=lens[:, None] - 1)[..., None]
    o = _attend(q, k.unsqueeze(2), v.unsqueeze(2), seen[:, None, None], st["scale"])
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)                              # [B, M, Hq, 256]
    return o[i < rows[:, None]].to(torch.bfloat16)


def _plain_prep(st):
    new, computed, T = st["new"].clamp(min=0), st["computed"], st["tokens"]
    S, dev = new.numel(), new.device
    lens = torch.where(new > 0, computed + new, 0)
    starts = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)]).to(torch.int32)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(starts, t.to(torch.int32), right=True) - 1
    live = t < starts[-1]
    seq = seq.clamp(max=S - 1)
    pos = torch.where(live, computed[seq] + (t - starts[seq]), -1).to(torch.int32)
    slots, taken, tables = [], [], []
    for table, bs, free in zip(st["tables"], st["sizes"], st["free"]):
        have, need = (computed + bs - 1) // bs, (lens + bs - 1) // bs
        count = torch.where(new > 0, need - have, 0)
        first = torch.cumsum(count, 0) - count
        col = torch.arange(table.shape[1], device=dev)
        fresh = (col >= have[:, None]) & (col < (have + count)[:, None])
        at = (first[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)
        table.copy_(torch.where(fresh, free[at.long()], table))
        page = table[seq, (pos // bs).clamp(min=0).long()].long()
        slots.append(torch.where(live, page * bs + pos % bs, -1))
        taken.append(count.sum().to(torch.int32))
        tables.append(table)
    return {"seq_lens": lens.to(torch.int32), "query_start_loc": starts, "positions": pos,
            "seq_idx": torch.where(live, seq, -1).to(torch.int32), "slots": slots,
            "taken": torch.stack(taken), "tables": tables}


def _plain_rope(st):
    def normed(x, w):
        x = x.float()
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    def turned(x):
        row = st["cos_sin"][st["positions"].long()].unsqueeze(1)
        rot = row.shape[-1]
        c, s = row[..., :rot // 2], row[..., rot // 2:]
        if st["neighbours"]:
            a, b = x[..., :rot:2], x[..., 1:rot:2]
            head = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            head = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([head, x[..., rot:]], -1).to(torch.bfloat16)

    st["k_cache"].flatten(0, 1)[st["slots"]] = turned(normed(st["k"], st["k_weight"]))
    st["v_cache"].flatten(0, 1)[st["slots"]] = st["v"]
    return turned(normed(st["q"], st["q_weight"])), st["k_cache"], st["v_cache"]


def _plain_write(st):
    slots, bs, got = st["slots"], st["bs"], []
    page, at = slots // bs, slots % bs
    for x, cache in ((st["key"], st["k_cache"]), (st["value"], st["v_cache"])):
        codes, s, lo = _quantised(x)
        rows = cache[..., :bs * 128].unflatten(-1, (bs, 128))
        pairs = cache[..., bs * 128:].unflatten(-1, (bs, 16))
        rows[page, :, at] = _rows(codes.transpose(0, 1), at).transpose(0, 1)
        pairs[page, :, at] = torch.stack([s, lo], -1).flatten(-2).view(torch.uint8)
        b = torch.gather(rows[page, :, at].unflatten(-1, (8, 16)), 2,
                         (torch.arange(8, device=x.device) ^ (at % 8)[:, None])[:, None, :, None]
                         .expand(-1, x.shape[1], -1, 16)).unflatten(-1, (GROUPS, 4))
        n = torch.stack([b & 15, b >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-2).float()
        pair = pairs[page, :, at].contiguous().view(torch.bfloat16).unflatten(-1, (GROUPS, 2)).float()
        got.append((pair[..., 1:] + pair[..., :1] * n).flatten(-2).to(torch.bfloat16))
    return got


# ------------------------------------------------------------------------------ the calls
def _own(st):
    import paged_kv_cache_09_gb300 as pa
    op = st["op"]
    if op == "prep":
        got = pa.batch_input_prep(st["computed"], st["new"], st["tables"], st["sizes"], st["free"],
                                  st["tokens"], out=st.get("out"))
        st["out"] = got
        return {"seq_lens": got["seq_lens"], "query_start_loc": got["query_start_loc"],
                "positions": got["positions"], "seq_idx": got["seq_idx"],
                "slots": got["slot_mappings"], "taken": got["pages_taken"], "tables": st["tables"]}
    if op == "rope":
        q = pa.qk_norm_rope_cache(st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"],
                                  st["cos_sin"], st["positions"], EPS, st["k_cache"], st["v_cache"],
                                  st["slots"], interleaved=st["neighbours"])
        return q, st["k_cache"], st["v_cache"]
    if op == "write":
        pa.reshape_and_cache_q4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["slots"])
        return list(pa.gather_cache_q4(st["k_cache"], st["v_cache"], st["slots"]))
    if op == "decode":
        if "workspace" not in st:
            need = pa.decode_q4_workspace_size(*st["q"].shape[:2], st["k_cache"].shape[1], D,
                                               st["bs"], st["longest"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return pa.decode_q4(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                            st["scale"], st["longest"], workspace=st["workspace"])
    if "workspace" not in st:
        need = pa.prefill_varlen_q4_workspace_size(st["starts"], st["lens"], True, st["q"].shape[1],
                                                   st["k_cache"].shape[1], D, st["bs"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return pa.prefill_varlen_q4(st["q"], st["k_cache"], st["v_cache"], st["table"], st["starts"],
                                st["lens"], True, st["scale"], workspace=st["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"prep": _plain_prep, "rope": _plain_rope, "write": _plain_write,
            "decode": _plain_decode, "prefill": _plain_prefill}[state["op"]](state)


# ------------------------------------------------------------------------------ what it takes
def work(case):
    op = case["op"]
    if op == "prep":
        S, T, sizes = case["seqs"], case["tokens"], [b for b in (case["bs0"], case["bs1"]) if b]
        # Lengths in, lengths and offsets out, positions, owners and slots out, new pages.
        pages = sum(T // b + S for b in sizes)
        return {"bytes": 8 * S + 8 * S + T * (8 + 8 * len(sizes)) + 8 * pages, "flops": 0}
    if op == "rope":
        rows = case["tokens"] * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 4 * rows * case["dim"] + case["tokens"] * (4 * case["rotary"] + 12),
                "flops": 8 * rows * case["dim"]}
    if op == "write":
        rows = 2 * case["tokens"] * case["hkv"]
        return {"bytes": rows * (2 * 2 * D + 2 * ROW_BYTES) + 8 * case["tokens"],
                "flops": 8 * rows * D}
    if op == "decode":
        keys = case["seqs"] * (case["low"] + case["high"]) / 2
        return {"bytes": keys * case["hkv"] * 2 * ROW_BYTES + 4 * case["seqs"] * case["hq"] * D,
                "flops": 4 * D * case["hq"] * keys}
    flops = data = 0
    for q, k in _chunks(case):
        flops += 4 * D * case["hq"] * (q * (k - q) + q * (q + 1) // 2)
        data += k * case["hkv"] * 2 * ROW_BYTES + 4 * q * case["hq"] * D
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------------------ in 64 bits
def _row64(cache, page, offset, bs):
    """The values of the tokens at `offset` of `page` [N]: fp64 [N, kv heads, 256], dim by
    dim from the format's description."""
    d = torch.arange(D, device=cache.device)
    group, unit, nibble = d // 64, d % 64 // 8, d % 8
    byte = offset[:, None] * 128 + (unit ^ (offset[:, None] % 8)) * 16 + group * 4 + nibble // 2
    flat = cache[page]                                                     # [N, heads, page bytes]
    raw = torch.gather(flat, 2, byte[:, None].expand(-1, flat.shape[1], -1))
    n = torch.div(raw, torch.where(nibble % 2 == 1, 16, 1), rounding_mode="floor") % 16
    base = bs * 128 + offset[:, None] * 16 + group * 4

    def bf16(first):
        low, high = (torch.gather(flat, 2, (base + first + i)[:, None].expand(-1, flat.shape[1], -1))
                     .to(torch.int32) for i in (0, 1))
        return ((low + (high << 8)) << 16).view(torch.float32).double()

    return bf16(2) + bf16(0) * n.double()


def _keys64(st, name, s, count):
    t = torch.arange(count, device="cuda")
    page = st["table"][s, t // st["bs"]].long()
    return torch.cat([_row64(st[name], p, o, st["bs"])
                      for p, o in zip(page.split(64), (t % st["bs"]).split(64))])


def _softmax64(q, k, v, scale, first):
    """q [M, Hq, 256] at positions first.. over k, v [N, Hkv, 256]."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // k.shape[1]
    pos = first + torch.arange(q.shape[0], device="cuda")
    hidden = torch.arange(k.shape[0], device="cuda") > pos[:, None]
    for h in range(q.shape[1]):
        w = torch.softmax((q[:, h].double() @ k[:, h // G].T * scale).masked_fill_(hidden, -math.inf), -1)
        out[:, h] = w @ v[:, h // G]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "prep":
        return None  # whole numbers only
    st = prepare(case, seed)
    if op == "rope":
        dim, rot = case["dim"], case["rotary"]
        half = rot // 2
        i = torch.arange(dim, device="cuda")
        if st["neighbours"]:
            other, freq, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0)
        else:
            other, freq, sign = (i + half) % rot, i % half, torch.where(i < half, -1.0, 1.0)
        turns = i < rot
        other, freq = torch.where(turns, other, i), torch.where(turns, freq, 0)
        table = st["cos_sin"].double()[st["positions"].long()]
        cos = torch.where(turns, table[:, freq], 1.0).unsqueeze(1)
        sin = torch.where(turns, table[:, half + freq] * sign, 0.0).unsqueeze(1)

        def turned(x, w):
            x = x.double()
            y = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / dim + EPS) * w.double()
            return y * cos + y[..., other] * sin

        k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
        page, at = st["slots"] // case["bs"], st["slots"] % case["bs"]
        k_cache[page, at] = turned(st["k"], st["k_weight"])
        v_cache[page, at] = st["v"].double()
        return turned(st["q"], st["q_weight"]), k_cache, v_cache
    if op == "write":
        got = []
        for x in (st["key"].double(), st["value"].double()):
            parts = []
            for g in range(GROUPS):
                y = x[..., 64 * g:64 * g + 64]
                lo = y.min(-1, keepdim=True).values
                s = ((y.max(-1, keepdim=True).values - lo) / 15).float().to(torch.bfloat16).double()
                parts.append(lo + s * ((y - lo) / s).round().clamp(max=15))
            got.append(torch.cat(parts, -1))
        return got
    if op == "decode":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        for s, n in enumerate(st["lens"].tolist()):
            k, v = (_keys64(st, c, s, n) for c in ("k_cache", "v_cache"))
            out[s] = _softmax64(st["q"][s:s + 1], k, v, st["scale"], n - 1)[0]
        return out
    parts = []
    for s, n in enumerate(st["lens"]):
        k, v = (_keys64(st, c, s, n) for c in ("k_cache", "v_cache"))
        q = st["q"][st["starts"][s]:st["starts"][s + 1]]
        parts.append(_softmax64(q, k, v, st["scale"], n - q.shape[0]))
    return torch.cat(parts)
