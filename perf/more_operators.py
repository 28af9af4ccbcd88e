"""Cases and plain forms of the 8-bit KV cache and of rotation by several axes.

Four operators, as a serving step uses them:

* ``mrope``    qk_norm_mrope_cache: RMS norm of each query and key head, rotation by a
               token's positions on several axes (time, height, width) and the KV write;
* ``write8``   reshape_and_cache_q8, then gather_cache_q8: new tokens quantised into the
               8-bit cache, and their blocks read back;
* ``decode8``  decode_q8: one query token per sequence over the 8-bit cache;
* ``prefill8`` prefill_varlen_q8: chunks of query rows over the 8-bit cache.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits.

The 8-bit cache.  Codes are e4m3 [pages, block_size, kv heads, 256], scales one byte for
each block of 16 tokens of a page and KV head, [pages, ceil(block_size / 16), kv heads]; a
code c under the byte b stands for c * 2^(b - 127) (255: NaN).  A write sets the byte of
each block that it touches to the smallest that keeps its new values within 448 * 2^(b - 127)
and is not below the present one.  Where it grows, the block's other rows are rounded to the new
scale.  Writing a block's first row begins it anew: the present byte and the rows that
are not written count no more.
"""
import math

import torch

own = False

D = 256
BLOCK = 16   # tokens of a scale
EPS = 1e-6


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # One layer's query/key step of a decode batch of 16 whose requests hold images:
        # quarter rotation, frequencies in three runs.
        {"name": "mrope 16 tokens", "op": "mrope", "tokens": 16, "hq": 24, "hkv": 4, "dim": 256,
         "rotary": 64, "pairs": "halves", "axes": "runs", "bs": 832, "table": 32768},
        # The same step of a q=4096 prompt chunk of text and image patches.
        {"name": "mrope 4096 tokens", "op": "mrope", "tokens": 4096, "hq": 24, "hkv": 4, "dim": 256,
         "rotary": 256, "pairs": "halves", "axes": "runs", "bs": 832, "table": 16384},
        # A shorter chunk, axes in turn from frequency to frequency.
        {"name": "mrope 1000 tokens in turn", "op": "mrope", "tokens": 1000, "hq": 32, "hkv": 8,
         "dim": 128, "rotary": 128, "pairs": "halves", "axes": "turns", "bs": 64, "table": 16384},
        # The new tokens of a decode batch of 16, most of them inside a block.
        {"name": "write8 16x1 tokens", "op": "write8", "seqs": 16, "new": 1, "low": 0, "high": 4096,
         "hkv": 4, "bs": 832},
        # The K/V of a q=4096 prompt chunk.
        {"name": "write8 1x4096 tokens", "op": "write8", "seqs": 1, "new": 4096, "low": 4096,
         "high": 4096, "hkv": 4, "bs": 832},
        # Several prompts' uneven chunks behind earlier tokens, small pages.
        {"name": "write8 12x333 tokens", "op": "write8", "seqs": 12, "new": 333, "low": 0,
         "high": 2000, "hkv": 8, "bs": 64},
        # A short single request: latency.
        {"name": "decode8 1x1701", "op": "decode8", "seqs": 1, "low": 1701, "high": 1701, "hq": 24,
         "hkv": 4, "bs": 832},
        # A single request at the longest context.
        {"name": "decode8 1x32768", "op": "decode8", "seqs": 1, "low": 32768, "high": 32768,
         "hq": 24, "hkv": 4, "bs": 832},
        # A decode batch of long, uneven contexts.
        {"name": "decode8 16x4096..32768", "op": "decode8", "seqs": 16, "low": 4096, "high": 32768,
         "hq": 24, "hkv": 4, "bs": 832},
        # Many short requests in small pages, another head layout.
        {"name": "decode8 64x1..2048 pages of 16", "op": "decode8", "seqs": 64, "low": 1,
         "high": 2048, "hq": 32, "hkv": 8, "bs": 16},
        # A prompt's last, shorter chunk over its earlier tokens.
        {"name": "prefill8 1685 over 12288", "op": "prefill8", "q0": 1685, "k0": 13973, "q1": 0,
         "k1": 0, "q2": 0, "k2": 0, "hq": 24, "hkv": 4, "bs": 832},
        # A mixed batch: a full chunk, a short one and a request of a few rows.
        {"name": "prefill8 mixed", "op": "prefill8", "q0": 4096, "k0": 8192, "q1": 512, "k1": 512,
         "q2": 5, "k2": 2999, "hq": 24, "hkv": 4, "bs": 784},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["mrope", "write8", "decode8", "decode8", "prefill8"])
    hq, hkv = rng.choice([(24, 4), (24, 4), (32, 8), (16, 2), (8, 8), (5, 1), (12, 4)])
    bs = rng.choice([16, 64, 784, 832, 7])
    if op == "mrope":
        dim = rng.choice([256, 256, 128, 64])
        return {"op": op, "tokens": _log(rng, 1, 4096), "hq": hq, "hkv": hkv, "dim": dim,
                "rotary": rng.choice([r for r in (16, 32, 64, 128, 256) if r <= dim]),
                "pairs": rng.choice(["halves", "neighbours"]),
                "axes": rng.choice(["runs", "turns"]), "bs": bs, "table": _log(rng, 8192, 262144)}
    if op == "write8":
        seqs = _log(rng, 1, 256)
        high = _log(rng, 1, 4096)
        return {"op": op, "seqs": seqs, "new": _log(rng, 1, max(1, 4096 // seqs)),
                "low": rng.choice([0, high]), "high": high, "hkv": min(hkv, 4), "bs": bs}
    if op == "decode8":
        seqs = _log(rng, 1, 64)
        high = _log(rng, 1, min(32768, 262144 * 4 // (seqs * max(hkv, 4))))
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


def _byte_for(top):
    """The smallest scale byte (1 at least) with top <= 448 * 2^(byte - 127): 448 is 0.875 * 2^9."""
    m, e = torch.frexp(top.float())
    return torch.where(top > 0, e - 9 + (m > 0.875).int() + 127, 1).clamp(1, 254)


def _power(e):
    """2^e, fp32; 0 below the normal range."""
    return ((e + 127).clamp(min=0).int() << 23).view(torch.float32)


def _filled(pool, hkv, bs, gen, peaked):
    """A whole pool of 8-bit pages of N(0, 1) rows: codes as bytes and scales; 5% of a key
    cache's rows eight times as large."""
    nb = -(-bs // BLOCK)
    codes = torch.empty((pool, bs, hkv, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pool, nb, hkv), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (hkv * bs * D))
    for p in range(0, pool, step):
        x = torch.randn((min(step, pool - p), bs, hkv, D), generator=gen, device="cuda")
        if peaked:
            x *= 1 + 7 * (torch.rand(x.shape[:3], generator=gen, device="cuda") < 0.05)[..., None]
        x = x.to(torch.bfloat16).float()
        top = torch.zeros((x.shape[0], nb * BLOCK, hkv), device="cuda")
        top[:, :bs] = x.abs().amax(-1)
        b = _byte_for(top.unflatten(1, (nb, BLOCK)).amax(2))
        rows = b.repeat_interleave(BLOCK, 1)[:, :bs, :, None]
        codes[p:p + step] = (x * _power(127 - rows)).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + step] = b.to(torch.uint8)
    return codes, scales


def _spoil_tails(codes, scales, table, lens, bs):
    """The last pages' places past each sequence's end hold NaN, as do scales of whole blocks."""
    for s, n in enumerate(lens):
        r = n % bs
        if r:
            page = int(table[s, n // bs])
            codes[page, r:] = 127
            scales[page, -(-r // BLOCK):] = 255


def _chunks(case):
    return [(case["q%d" % i], case["k%d" % i]) for i in range(3) if case["k%d" % i]]


def _axis_of(half, how):
    """Axis of each frequency: half of them time, a quarter each height and width, in three
    runs or in turn."""
    h = half // 4
    if how == "runs":
        return [0] * (half - 2 * h) + [1] * h + [2] * h
    return [i % 3 if i % 3 and i // 3 < h else 0 for i in range(half)]


def _positions(tokens, table, gen):
    """int32 [3, tokens]: stretches of text (all axes alike) and of image patches in rows."""
    t = torch.arange(tokens, device="cuda")
    side = int(_pick(4, 40, 1, gen))
    span = side * side + 37                       # 37 text tokens, then an image
    image, at = t // span, t % span - 37
    text = at < 0
    base = image * (37 + side)                    # an image takes `side` positions of each axis
    pos = torch.stack([base + torch.where(text, at + 37, 37),
                       base + torch.where(text, at + 37, 37 + at // side),
                       base + torch.where(text, at + 37, 37 + at % side)])
    first = int(_pick(0, max(0, table - int(pos.max()) - 1), 1, gen))
    return (pos + first).clamp(max=table - 1).to(torch.int32)


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "mrope":
        T, hq, hkv, dim, bs = (case[k] for k in ("tokens", "hq", "hkv", "dim", "bs"))
        packed = _normal((T, (hq + 2 * hkv) * dim), gen)  # the projection's output
        q, k, v = (x.unflatten(1, (-1, dim)) for x in packed.split([hq * dim, hkv * dim, hkv * dim], 1))
        rot = case["rotary"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * freq
        pool = -(-T // bs) + 2
        weight = [(1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).to(torch.bfloat16)
                  for _ in range(2)]
        slots = torch.randperm(pool, generator=gen, device="cuda")[torch.arange(T, device="cuda") // bs]
        return {"op": op, "q": q, "k": k, "v": v, "q_weight": weight[0], "k_weight": weight[1],
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
                "neighbours": case["pairs"] == "neighbours", "axes": _axis_of(rot // 2, case["axes"]),
                "positions": _positions(T, case["table"], gen),
                "slots": slots * bs + torch.arange(T, device="cuda") % bs,
                "k_cache": _normal((pool, bs, hkv, dim), gen),
                "v_cache": _normal((pool, bs, hkv, dim), gen)}
    hkv, bs = case["hkv"], case["bs"]
    if op == "write8":
        S, n = case["seqs"], case["new"]
        old = _pick(case["low"], case["high"], S, gen).tolist()
        table, pool = _tables([c + n for c in old], bs, 2, gen)
        wide = table.long()

        def slots_of(s, first, last):
            t = torch.arange(first, last, device="cuda")
            return wide[s, t // bs] * bs + t % bs

        # Behind the earlier tokens, the new ones; what is read back: their blocks' tokens, behind
        # padding where the first block holds fewer than 15 earlier ones.
        def back_of(s, c):
            held = c % bs % BLOCK
            return torch.cat([wide.new_full((BLOCK - 1 - held,), -1), slots_of(s, c - held, c + n)])

        state = {"op": op, "bs": bs,
                 "slots": torch.cat([slots_of(s, c, c + n) for s, c in enumerate(old)]),
                 "back": torch.cat([back_of(s, c) for s, c in enumerate(old)]),
                 "key": _normal((S * n, hkv, D), gen), "value": _normal((S * n, hkv, D), gen)}
        loud = 1 + 7 * (torch.rand((S * n, hkv, 1), generator=gen, device="cuda") < 0.05)
        state["key"] *= loud.to(torch.bfloat16)
        for name in ("k", "v"):
            codes, scales = _filled(pool, hkv, bs, gen, name == "k")
            _spoil_tails(codes, scales, table, old, bs)
            state[name + "_cache"], state[name + "_scales"] = codes.view(torch.float8_e4m3fn), scales
        return state
    hq = case["hq"]
    if op == "decode8":
        lens = _pick(case["low"], case["high"], case["seqs"], gen)
        lens[0] = case["high"]
        lens = lens.tolist()
    else:
        lens = [k for _, k in _chunks(case)]
    table, pool = _tables(lens, bs, 3, gen)
    state = {"op": op, "table": table, "bs": bs, "scale": 1.0 / math.sqrt(D)}
    for name in ("k", "v"):
        codes, scales = _filled(pool, hkv, bs, gen, name == "k")
        _spoil_tails(codes, scales, table, lens, bs)
        state[name + "_cache"], state[name + "_scales"] = codes.view(torch.float8_e4m3fn), scales
    if op == "decode8":
        return {**state, "q": _normal((len(lens), hq, D), gen), "longest": max(lens),
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    starts = [0]
    for q, _ in _chunks(case):
        starts.append(starts[-1] + q)
    return {**state, "q": _normal((starts[-1], hq, D), gen), "starts": starts, "lens": lens}


# ------------------------------------------------------------------------------ plain forms
def _sequences(codes, scales, table, bs):
    """Every sequence's values, fp32 [S, kv heads, pages * block_size, 256]."""
    at = table.clamp(min=0).long()
    b = scales[at].repeat_interleave(BLOCK, 2)[:, :, :bs].int()
    x = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x = torch.where(b.unsqueeze(-1) == 255, math.nan, x * _power(b - 127).unsqueeze(-1))
    return x.flatten(1, 2).transpose(1, 2)


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
    hkv = st["k_cache"].shape[2]
    k, v = (_sequences(st[n + "_cache"], st[n + "_scales"], st["table"], st["bs"]) for n in "kv")
    seen = (torch.arange(k.shape[2], device="cuda") < st["lens"][:, None])[:, None, None]
    q = st["q"].float().view(S, hkv, hq // hkv, D)
    return _attend(q, k, v, seen, st["scale"]).view(S, hq, D).to(torch.bfloat16)


def _plain_prefill(st):
    """Every chunk padded to the longest one."""
    total, hq, _ = st["q"].shape
    hkv, dev = st["k_cache"].shape[2], st["q"].device
    k, v = (_sequences(st[n + "_cache"], st[n + "_scales"], st["table"], st["bs"]) for n in "kv")
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


def _plain_rope(st):
    def normed(x, w):
        x = x.float()
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    axis = torch.tensor(st["axes"], device="cuda")
    half = axis.numel()
    at = st["positions"].long()[axis].T                                   # [T, half]
    i = torch.arange(half, device="cuda")
    c, s = (st["cos_sin"][at, i + o].unsqueeze(1) for o in (0, half))

    def turned(x):
        if st["neighbours"]:
            a, b = x[..., :2 * half:2], x[..., 1:2 * half:2]
            head = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            head = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([head, x[..., 2 * half:]], -1).to(torch.bfloat16)

    st["k_cache"].flatten(0, 1)[st["slots"]] = turned(normed(st["k"], st["k_weight"]))
    st["v_cache"].flatten(0, 1)[st["slots"]] = st["v"]
    return turned(normed(st["q"], st["q_weight"])), st["k_cache"], st["v_cache"]


def _plain_write(st):
    slots, bs, got = st["slots"], st["bs"], []
    nb = st["k_scales"].shape[1]
    block = slots // bs * nb + slots % bs // BLOCK
    touched, mine = torch.unique(block, return_inverse=True)
    begun = torch.zeros(touched.numel(), dtype=torch.bool, device="cuda")
    begun[mine[slots % bs % BLOCK == 0]] = True
    row = torch.arange(BLOCK, device="cuda")
    inside = (touched % nb * BLOCK)[:, None] + row < bs                   # rows that the page has
    places = ((touched // nb * bs + touched % nb * BLOCK)[:, None] + row)
    for n, x in (("k", st["key"]), ("v", st["value"])):
        codes = st[n + "_cache"].view(torch.uint8).flatten(0, 1)          # [slots, heads, 256]
        scales = st[n + "_scales"].flatten(0, 1)                          # [blocks, heads]
        x = x.float()
        need = torch.zeros((touched.numel(), x.shape[1]), dtype=torch.int32, device="cuda")
        need.scatter_reduce_(0, mine[:, None].expand(-1, x.shape[1]), _byte_for(x.abs().amax(-1)), "amax")
        old = scales[touched].int()
        old = torch.where(begun[:, None] | (old == 255), 0, old)
        new = torch.maximum(old, need)
        move = inside & ~begun[:, None]
        at, who = places[move], torch.arange(touched.numel(), device="cuda")[:, None].expand(-1, BLOCK)[move]
        was = codes[at].view(torch.float8_e4m3fn).float()
        codes[at] = (was * _power(old - new)[who].unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[slots] = (x * _power(127 - new)[mine].unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[touched] = new.to(torch.uint8)
        back = st["back"].clamp(min=0)
        b = scales[back // bs * nb + back % bs // BLOCK].int()
        c = codes[back].view(torch.float8_e4m3fn).float()
        value = (c * _power(b - 127).unsqueeze(-1)).to(torch.bfloat16)
        got.append(value.masked_fill((st["back"] < 0)[:, None, None], 0))
    return got


# ------------------------------------------------------------------------------ the calls
def _own(st):
    import paged_kv_cache_09_gb300 as pa
    op = st["op"]
    if op == "mrope":
        if not isinstance(st["axes"], bytes):
            st["axes"] = bytes(st["axes"])
        q = pa.qk_norm_mrope_cache(st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"],
                                   st["cos_sin"], st["positions"], st["axes"], EPS, st["k_cache"],
                                   st["v_cache"], st["slots"], interleaved=st["neighbours"])
        return q, st["k_cache"], st["v_cache"]
    cache = (st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"])
    if op == "write8":
        pa.reshape_and_cache_q8(st["key"], st["value"], *cache, st["slots"])
        return list(pa.gather_cache_q8(*cache, st["back"]))
    if op == "decode8":
        if "workspace" not in st:
            need = pa.decode_q8_workspace_size(*st["q"].shape[:2], st["k_cache"].shape[2], D,
                                               st["bs"], st["longest"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return pa.decode_q8(st["q"], *cache, st["table"], st["lens"], st["scale"], st["longest"],
                            workspace=st["workspace"])
    if "workspace" not in st:
        need = pa.prefill_varlen_q8_workspace_size(st["starts"], st["lens"], True, st["q"].shape[1],
                                                   st["k_cache"].shape[2], D, st["bs"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return pa.prefill_varlen_q8(st["q"], *cache, st["table"], st["starts"], st["lens"], True,
                                st["scale"], workspace=st["workspace"])


def run(state):
    if own:
        return _own(state)
    return {"mrope": _plain_rope, "write8": _plain_write, "decode8": _plain_decode,
            "prefill8": _plain_prefill}[state["op"]](state)


# ------------------------------------------------------------------------------ what it takes
def work(case):
    op = case["op"]
    if op == "mrope":
        rows = case["tokens"] * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 4 * rows * case["dim"] + case["tokens"] * (4 * case["rotary"] + 20),
                "flops": 8 * rows * case["dim"]}
    if op == "write8":
        # New rows in and their codes out; codes of their blocks in and the rows out.
        new = case["seqs"] * case["new"]
        back = new + case["seqs"] * (BLOCK - 1)
        rows = 2 * case["hkv"]
        return {"bytes": rows * D * (3 * new + 3 * back) + rows * (new + back) // 8 + 8 * (new + back),
                "flops": 4 * rows * D * new}
    row = 2 * (D + 1.0 / BLOCK)  # a key's codes and its share of the scales, of K and V
    if op == "decode8":
        keys = case["seqs"] * (case["low"] + case["high"]) / 2
        return {"bytes": keys * case["hkv"] * row + 4 * case["seqs"] * case["hq"] * D,
                "flops": 4 * D * case["hq"] * keys}
    flops = data = 0
    for q, k in _chunks(case):
        flops += 4 * D * case["hq"] * (q * (k - q) + q * (q + 1) // 2)
        data += k * case["hkv"] * row + 4 * q * case["hq"] * D
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------------------ in 64 bits
def _power64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decoded64(byte):
    """e4m3 bytes -> fp64, from the bits: sign, 4 of exponent (bias 7), 3 of fraction."""
    b = byte.to(torch.int32)
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (8 + f) * _power64(e - 10), f * 2.0 ** -9)
    mag = torch.where((b & 127) == 127, math.nan, mag)
    return torch.where(b > 127, -mag, mag)


def _rounded64(x):
    """fp64 (within 448) -> the nearest e4m3 values, ties to even."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4          # 2^e: a step of x's binade
    return torch.round(x * _power64(-e)) * _power64(e)


def _keys64(st, name, s, count):
    t = torch.arange(count, device="cuda")
    page, at = st["table"][s, t // st["bs"]].long(), t % st["bs"]
    codes = st[name + "_cache"].view(torch.uint8)[page, at]
    exp = st[name + "_scales"][page, torch.div(at, BLOCK, rounding_mode="floor")].to(torch.int32)
    return _decoded64(codes) * _power64(exp - 127).unsqueeze(-1)


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


def _write64(st):
    """Block by block: the block's values after the write, then what is read back."""
    bs, blocks, got = st["bs"], {}, []
    for t, s in enumerate(st["slots"].tolist()):
        blocks.setdefault((s // bs, s % bs // BLOCK), {})[s % bs % BLOCK] = t
    for n, x in (("k", st["key"].double()), ("v", st["value"].double())):
        codes, scales = st[n + "_cache"].view(torch.uint8), st[n + "_scales"].cpu()
        loudest, after = x.abs().amax(-1).cpu(), {}
        for (page, i), rows in blocks.items():
            tokens, places = torch.tensor(list(rows.values())), torch.tensor(list(rows), device="cuda")
            top = loudest[tokens].amax(0)                                  # [heads]
            exp = torch.ceil(torch.log2(top / 448))
            exp = torch.where(top > 448 * 2.0 ** exp, exp + 1, exp)
            exp = torch.where(top <= 448 * 2.0 ** (exp - 1), exp - 1, exp).clamp(min=-126)
            old = scales[page, i].double() - 127
            if 0 not in rows:
                exp = torch.where(old < 128, torch.maximum(exp, old), exp)
            unit = (2.0 ** exp).cuda()[:, None]
            part = _decoded64(codes[page, i * BLOCK:(i + 1) * BLOCK])      # [rows, heads, 256]
            part = _rounded64(part * (2.0 ** (old - exp)).cuda()[:, None]) * unit
            part[places] = _rounded64(x[tokens.cuda()] / unit) * unit
            after[page, i] = part
        got.append(torch.stack([after[s // bs, s % bs // BLOCK][s % bs % BLOCK] if s >= 0
                                else x.new_zeros(x.shape[1:]) for s in st["back"].tolist()]))
    return got


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "mrope":
        dim, rot = case["dim"], case["rotary"]
        half = rot // 2
        i = torch.arange(dim, device="cuda")
        if st["neighbours"]:
            other, freq, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0)
        else:
            other, freq, sign = (i + half) % rot, i % half, torch.where(i < half, -1.0, 1.0)
        turns = i < rot
        other, freq = torch.where(turns, other, i), torch.where(turns, freq, 0)
        place = torch.stack([st["positions"][a] for a in st["axes"]], 1).long()[:, freq]
        cos = torch.where(turns, st["cos_sin"].double()[place, freq], 1.0).unsqueeze(1)
        sin = torch.where(turns, st["cos_sin"].double()[place, half + freq] * sign, 0.0).unsqueeze(1)

        def turned(x, w):
            x = x.double()
            y = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / dim + EPS) * w.double()
            return y * cos + y[..., other] * sin

        k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
        page, at = st["slots"] // case["bs"], st["slots"] % case["bs"]
        k_cache[page, at] = turned(st["k"], st["k_weight"])
        v_cache[page, at] = st["v"].double()
        return turned(st["q"], st["q_weight"]), k_cache, v_cache
    if op == "write8":
        return _write64(st)
    if op == "decode8":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        for s, n in enumerate(st["lens"].tolist()):
            k, v = (_keys64(st, c, s, n) for c in "kv")
            out[s] = _softmax64(st["q"][s:s + 1], k, v, st["scale"], n - 1)[0]
        return out
    parts = []
    for s, n in enumerate(st["lens"]):
        k, v = (_keys64(st, c, s, n) for c in "kv")
        q = st["q"][st["starts"][s]:st["starts"][s + 1]]
        parts.append(_softmax64(q, k, v, st["scale"], n - q.shape[0]))
    return torch.cat(parts)
