"""Serving from a cache held in 8 bits, and with a window over long contexts: what is measured, and its plain form.

Three operators of a serving step: rotary positions with the write into a paged cache of 8-bit
values ("append8"), attention of new tokens over that cache ("attn8"), and attention that sees a
sliding window and a few first tokens, over a cache of 16- or 32-bit values ("window") or over the
8-bit one (an "attn8" case with a window).

The 8-bit cache holds e4m3 values and, for each block of tokens and head, a power of two.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGEST = 448.0  # of e4m3
LOWEST, HIGHEST = -110, 119  # the exponents that an append writes


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 sequences: the smallest call, into blocks that are part full
        dict(name="append8 decode", op="append8", dtype="bf16", seqs=8, q_min=1, q_max=1, past=900, heads=32,
             kv_heads=4, dim=128, rot=128, interleaved=False, norm=True, page=16, block=16, lens=1),
        # prompts of 3 requests prefilled in one call
        dict(name="append8 prompt", op="append8", dtype="bf16", seqs=3, q_min=1100, q_max=1700, past=0, heads=32,
             kv_heads=4, dim=128, rot=128, interleaved=False, norm=True, page=64, block=64, lens=2),
        # fp32, interleaved pairs on part of an odd head size, chunks behind what is cached, a scale a page of odd size
        dict(name="append8 part fp32", op="append8", dtype="f32", seqs=5, q_min=101, q_max=411, past=37, heads=12,
             kv_heads=3, dim=96, rot=64, interleaved=True, norm=False, page=24, block=24, lens=3),
        # one decode step of 8 sequences at short contexts
        dict(name="attn8 decode short", op="attn8", dtype="bf16", seqs=8, q_min=1, q_max=1, kv_min=90, kv_max=1100,
             heads=32, kv_heads=4, dim=128, page=16, block=16, window=0, sinks=0, lse=False, short=False, lens=4),
        # a full decode batch, ragged contexts of up to 16k tokens
        dict(name="attn8 decode batch", op="attn8", dtype="bf16", seqs=64, q_min=1, q_max=1, kv_min=500, kv_max=16000,
             heads=32, kv_heads=4, dim=128, page=64, block=64, window=0, sinks=0, lse=False, short=False, lens=5),
        # a single user at a very long context: the split over the cache decides
        dict(name="attn8 decode long", op="attn8", dtype="bf16", seqs=1, q_min=1, q_max=1, kv_min=131071,
             kv_max=131071, heads=32, kv_heads=4, dim=128, page=128, block=32, window=0, sinks=0, lse=True,
             short=False, lens=6),
        # a chunk of a long prompt over what is already cached: the largest call
        dict(name="attn8 chunk", op="attn8", dtype="bf16", seqs=1, q_min=2048, q_max=2048, kv_min=16384,
             kv_max=16384, heads=32, kv_heads=4, dim=128, page=64, block=64, window=0, sinks=0, lse=False,
             short=False, lens=8),
        # a mixed step with a window: chunks and single tokens, one sequence whose first rows see no key
        dict(name="attn8 mixed window", op="attn8", dtype="bf16", seqs=7, q_min=1, q_max=900, kv_min=5, kv_max=5000,
             heads=16, kv_heads=2, dim=64, page=32, block=16, window=1000, sinks=5, lse=True, short=True, lens=9),
        # a few tokens each (draft tokens to be checked), fp32 queries, odd head and page sizes, a scale a token
        dict(name="attn8 few fp32", op="attn8", dtype="f32", seqs=6, q_min=1, q_max=5, kv_min=3, kv_max=1500,
             heads=12, kv_heads=4, dim=80, page=10, block=1, window=700, sinks=3, lse=True, short=False, lens=7),
        # a full decode batch of a layer with a window, far into their contexts
        dict(name="window decode batch", op="window", dtype="bf16", seqs=64, q_min=1, q_max=1, kv_min=500,
             kv_max=16000, heads=32, kv_heads=4, dim=128, page=64, window=1024, sinks=4, lse=False, short=False,
             lens=10),
        # a single user at a very long context
        dict(name="window decode one", op="window", dtype="bf16", seqs=1, q_min=1, q_max=1, kv_min=70001,
             kv_max=70001, heads=32, kv_heads=4, dim=128, page=16, window=4097, sinks=1, lse=True, short=False,
             lens=11),
        # a chunk of a long prompt in a layer with a window
        dict(name="window chunk", op="window", dtype="bf16", seqs=1, q_min=2048, q_max=2048, kv_min=16384,
             kv_max=16384, heads=32, kv_heads=4, dim=128, page=64, window=4096, sinks=4, lse=False, short=False,
             lens=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= 5.0e8 and w["flops"] <= 2.5e11:
            return c


def _draw(rng):
    op = rng.choice(["append8", "attn8", "attn8", "window"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
    common = dict(heads=heads, kv_heads=kv_heads, lens=rng.randrange(1 << 30))
    if op == "append8":
        dim = rng.choice([64, 96, 128, 128, 256])
        q_max = rng.choice([1, _log(rng, 2, 1500)])
        page = rng.choice([16, 24, 64, 128])
        return dict(op="append8", dtype=rng.choice(["bf16", "bf16", "f32"]),
                    seqs=_log(rng, 1, 3) if q_max > 300 else _log(rng, 1, 12) if q_max > 1 else _log(rng, 1, 64),
                    q_min=1, q_max=q_max, past=rng.randrange(200), dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, page=page,
                    block=rng.choice([page, page, page // 2, 8]), **common)
    kind = rng.choice(["decode", "few", "chunk", "chunk"])
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    most = 2000 if dtype == "f32" else 20000
    kv_max = _log(rng, 20, most)
    if kind == "chunk":
        q_max = _log(rng, 8, 200 if dtype == "f32" else 1500)
        seqs = _log(rng, 1, 6)
    else:
        q_max = 1 if kind == "decode" else rng.randrange(2, 7)
        seqs = _log(rng, 1, 40)
    page = rng.choice([16, 32, 64, 128])
    windowed = op == "window" or rng.random() < 0.4
    c = dict(op=op, dtype=dtype, seqs=seqs, q_min=1, q_max=q_max, kv_min=max(1, kv_max // 20), kv_max=kv_max,
             dim=rng.choice([64, 128, 128]), page=page, window=_log(rng, 16, 5000) if windowed else 0,
             sinks=rng.choice([0, 1, 4, rng.randrange(150)]) if windowed else 0, lse=rng.random() < 0.5,
             short=q_max > 1 and rng.random() < 0.25, **common)
    if op == "attn8":
        c["block"] = rng.choice([16, 16, page, page // 2])
    return c


# ------------------------------------------------------------------------------- inputs

def _lengths(c):
    """The chunk and cache lengths of the case's sequences: lists, the same for every seed."""
    r = random.Random(c["lens"])
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["seqs"])]
    q[r.randrange(c["seqs"])] = c["q_max"]
    if c["op"] == "append8":
        return q, [n + r.randint(0, c["past"]) for n in q]
    kv = [r.randint(c["kv_min"], c["kv_max"]) for _ in range(c["seqs"])]
    kv[r.randrange(c["seqs"])] = c["kv_max"]
    kv = [max(n, m) for n, m in zip(q, kv)]  # a sequence's keys include its chunk's own
    if c["short"]:  # but for one, cut short: its first rows see no key
        i = r.randrange(c["seqs"])
        kv[i] = max(1, q[i] // 2)
    return q, kv


def _seen(c, n, m):
    """Of a chunk of n in a sequence of m keys: how many (token, key) pairs the mask lets through, and how many keys
    some token sees."""
    window, sinks = c["window"] or m, c["sinks"]
    pairs, first = 0, None
    for place in range(max(0, m - n), m):
        low = max(0, place + 1 - window)
        first = low if first is None else first
        pairs += place + 1 - low + min(low, sinks)
    return pairs, 0 if first is None else m - first + min(first, sinks)


def work(case):
    c = case
    q, kv = _lengths(c)
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "append8":
        q_values, kv_values = sum(q) * c["heads"] * c["dim"], sum(q) * 2 * c["kv_heads"] * c["dim"]
        blocks = sum(-(-m // c["block"]) - (m - n) // c["block"] for n, m in zip(q, kv))
        return {"bytes": 2 * q_values * size + kv_values * (size + 1) + blocks * 2 * c["kv_heads"],
                "flops": 6 * (q_values + kv_values)}
    pairs, keys = (sum(x) for x in zip(*(_seen(c, n, m) for n, m in zip(q, kv))))
    rows = sum(q) * c["heads"]
    values = 2 * keys * c["kv_heads"] * c["dim"]
    cache = values + 2 * (keys // c["block"]) * c["kv_heads"] if c["op"] == "attn8" else values * size
    return {"bytes": 2 * rows * c["dim"] * size + cache + 4 * rows * c["lse"],
            "flops": 4 * pairs * c["heads"] * c["dim"]}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _paging(c, kv, g):
    """Page numbers in a shuffled order, a row a sequence; what no sequence needs is -1."""
    need = [-(-n // c["page"]) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((len(kv), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _held(s, c, pages):
    """[pages][slots]: whether a sequence holds the slot."""
    slot = torch.arange(s["table"].shape[1] * c["page"], device=DEV).view(1, -1, c["page"])
    used = torch.zeros(pages, c["page"], dtype=torch.bool, device=DEV)
    mapped = s["table"] >= 0
    used[s["table"][mapped].long()] = (slot < s["kv_len"].view(-1, 1, 1))[mapped]
    return used


def _exponents(top):
    """The smallest e with top <= 448 * 2^e, within the range that is written; whole numbers."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, e, torch.full_like(e, LOWEST)).clamp(LOWEST, HIGHEST)


def _power(e):
    """2^e as fp32, put together from its bits."""
    return ((e.clamp(-126, 127) + 127) << 23).int().view(torch.float32)


def _cache8(c, pages, g, used):
    """Values with a spread that changes from block to block, as 8-bit codes and exponents; what no sequence has
    written is NaN."""
    shape = (pages, c["kv_heads"], c["page"] // c["block"], c["block"], c["dim"])
    x = torch.randn(shape, generator=g, device=DEV)
    x *= 0.7 + 0.6 * torch.rand(shape[:3] + (1, 1), generator=g, device=DEV)
    e = _exponents(x.abs().amax((3, 4)))
    codes = (x / _power(e)[..., None, None]).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).view(pages, c["kv_heads"], c["page"], c["dim"])
    codes.masked_fill_(~used.view(pages, 1, c["page"], 1), 0x7f)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    q_len, kv_len = _lengths(c)
    n, dt = sum(q_len), DTYPES[c["dtype"]]
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    s["table"], pages = _paging(c, kv_len, g)
    s["cu_q"] = torch.tensor([0] + q_len, device=DEV).cumsum(0).int()
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    s["q_max"], s["tokens"] = max(q_len), n
    used = _held(s, c, pages)
    if c["op"] == "append8":
        # q, k and v are slices of the projection's output
        qkv = torch.randn(n, (heads + 2 * kv_heads) * dim, generator=g, device=DEV).to(dt)
        q, k, v = qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], dim=1)
        s["q"], s["k"], s["v"] = q.view(n, heads, dim), k.view(n, kv_heads, dim), v.view(n, kv_heads, dim)
        s["q_out"] = torch.empty(n, heads, dim, dtype=dt, device=DEV)
        s["gq"], s["gk"] = ((1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(dt) if c["norm"] else None
                            for _ in range(2))
        for name in ("k", "v"):  # what is cached is smaller than what comes, so that some blocks' scales grow
            codes, e = _cache8(c, pages, g, used)
            s[name + "_codes"] = torch.where(used.view(pages, 1, c["page"], 1), codes, torch.zeros_like(codes))
            s[name + "_scale"] = e - torch.randint(0, 2, e.shape, generator=g, device=DEV, dtype=torch.uint8)
    else:
        # scores with a spread of about 1.5, as trained heads have
        s["q"] = (1.5 * torch.randn(n, heads, dim, generator=g, device=DEV)).to(dt)
        for name in ("k", "v"):
            if c["op"] == "attn8":
                s[name + "_codes"], s[name + "_scale"] = _cache8(c, pages, g, used)
            else:
                x = torch.randn(pages, kv_heads, c["page"], dim, generator=g, device=DEV).to(dt)
                s[name + "_cache"] = x.masked_fill_(~used.view(pages, 1, c["page"], 1), float("nan"))
        s["out"] = torch.empty(n, heads, dim, dtype=dt, device=DEV)
        s["lse"] = torch.empty(n, heads, dtype=torch.float32, device=DEV) if c["lse"] else None
        s["scale"] = 1 / math.sqrt(dim)
    if own:
        import top_routing_grouped_router_gb300 as moe
        s["shape"] = moe.make_attn_shape(n, c["seqs"], heads, kv_heads, dim, c["page"], pages, s["table"].shape[1],
                                         s["q_max"], act=c["dtype"])
        s["batch"] = moe.make_attn_batch(s["cu_q"], s["kv_len"], s["table"])
        if c["op"] == "window":
            s["cache"] = moe.make_kv_cache(s["k_cache"], s["v_cache"])
            size = moe.moe_attn_workspace_size(s["shape"])
        else:
            s["cache"] = moe.make_kv_cache_q8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
            size = moe.moe_attn_q8_workspace_size(s["shape"], c["block"])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
        if c["op"] == "append8":
            s["rope"] = moe.make_rope(c["rot"], base=1000000.0, interleaved=c["interleaved"], q_gamma=s["gq"],
                                      k_gamma=s["gk"], eps=1e-6)
        else:
            s["window"] = moe.make_attn_window(c["window"], c["sinks"]) if c["window"] else None
    return s


# ------------------------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import top_routing_grouped_router_gb300 as moe
        if op == "append8":
            moe.moe_rope_append_q8(s["shape"], s["rope"], s["q"], s["k"], s["v"], s["cache"], s["batch"], s["q_out"],
                                   workspace=s["ws"])
            return {"q": s["q_out"], **_cache_values(s)}
        if op == "attn8":
            moe.moe_paged_attention_q8(s["shape"], s["q"], s["cache"], s["batch"], s["out"], window=s["window"],
                                       scale=s["scale"], lse=s["lse"], workspace=s["ws"])
        else:
            moe.moe_paged_attention_window(s["shape"], s["q"], s["cache"], s["batch"], s["window"], s["out"],
                                           scale=s["scale"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    return _plain_append(s) if op == "append8" else _plain_attn(s)


def _cache_values(s):
    """The cache as it lies there, each byte as the value that it stands for: e4m3, and powers of two."""
    return {name + end: s[name + end].view(dt) for name in ("k", "v")
            for end, dt in (("_codes", torch.float8_e4m3fn), ("_scale", torch.float8_e8m0fnu))}


def _rows_of(s):
    """For each new token its sequence and its place in the sequence."""
    at = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(s["cu_q"], at.int(), right=True) - 1
    place = s["kv_len"][seq] - (s["cu_q"][seq + 1] - at)
    return seq, place


def _round8(x):
    """The nearest e4m3 values (ties to even), x within +-448; as fp32."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _plain_append(s):
    c = s["c"]
    block, page = c["block"], c["page"]
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    rates = torch.pow(torch.tensor(1000000.0, dtype=torch.float64, device=DEV), -2 * i / c["rot"])
    seq, place = _rows_of(s)
    angle = place.double().unsqueeze(1) * rates
    cos, sin = (f(angle).float().unsqueeze(1) for f in (torch.cos, torch.sin))

    def turn(x, gamma):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * gamma.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=3).flatten(2)
        else:
            a, b = r.chunk(2, dim=2)
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=2)
        return torch.cat((r, rest), dim=2)

    # the blocks that the chunks touch, numbered [page][block of the page]
    pages, kv_heads = s["k_codes"].shape[:2]
    per = page // block
    home = s["table"][seq, place // page].long() * per + place % page // block
    slot = place % block
    first = (s["kv_len"] - (s["cu_q"][1:] - s["cu_q"][:-1]))[seq]  # the chunk's first place
    kept = torch.where(place // block == first // block, first % block, torch.zeros_like(first))  # old tokens in the block
    old_in = torch.zeros(pages * per, dtype=torch.int64, device=DEV)
    old_in[home] = kept.long()
    touched = torch.zeros(pages * per, 1, dtype=torch.bool, device=DEV)
    touched[home] = True
    for name, x in (("k", turn(s["k"], s["gk"])), ("v", s["v"].float())):
        codes = s[name + "_codes"].view(torch.float8_e4m3fn).float().view(pages, kv_heads, per, block, c["dim"])
        codes = codes.transpose(1, 2).reshape(pages * per, kv_heads, block, c["dim"])
        was = s[name + "_scale"].int().transpose(1, 2).reshape(pages * per, kv_heads) - 127
        top = torch.zeros(pages * per, kv_heads, device=DEV)
        top.index_reduce_(0, home, x.abs().amax(2), "amax")
        e = _exponents(top)
        e = torch.where(old_in.unsqueeze(1) > 0, torch.maximum(e, was), e)
        old = torch.arange(block, device=DEV) < old_in.unsqueeze(1)  # [block number][slot]
        moved = _round8(codes * _power(was - e)[..., None, None])
        codes = torch.where((touched & old)[:, None, :, None], moved, codes)
        codes[home, :, slot] = _round8((x * _power(-e[home]).unsqueeze(2)).clamp(-LARGEST, LARGEST))
        e = torch.where(touched, e, was)
        codes = codes.view(pages, per, kv_heads, block, c["dim"]).transpose(1, 2)
        s[name + "_codes"].copy_(codes.reshape(pages, kv_heads, page, c["dim"]).to(torch.float8_e4m3fn).view(torch.uint8))
        s[name + "_scale"].copy_((e + 127).to(torch.uint8).view(pages, per, kv_heads).transpose(1, 2))
    return {"q": turn(s["q"], s["gq"]).to(DTYPES[c["dtype"]]), **_cache_values(s)}


def _plain_attn(s):
    c = s["c"]
    seqs, heads, kv_heads, dim = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    q_max, group = s["q_max"], heads // kv_heads
    seq, place = _rows_of(s)
    j = torch.arange(s["tokens"], device=DEV) - s["cu_q"][seq]
    # the chunks side by side, padded to the longest
    q = torch.zeros(seqs, q_max, heads, dim, device=DEV)
    q[seq, j] = s["q"].float()
    q = q.view(seqs, q_max, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv_heads, group * q_max, dim)
    # each sequence's pages in order
    table = s["table"].clamp(min=0).long()

    def rows(name):
        if c["op"] == "attn8":
            x = s[name + "_codes"][table].view(torch.float8_e4m3fn).float()
            x = x.unflatten(3, (-1, c["block"])) * _power(s[name + "_scale"][table].int() - 127)[..., None, None]
            x = x.flatten(3, 4)
        else:
            x = s[name + "_cache"][table].float()
        return x.permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, -1, dim)

    k, v = rows("k"), rows("v")
    key = torch.arange(k.shape[2], device=DEV)
    held = key < s["kv_len"].unsqueeze(1)
    k, v = (torch.where(held.view(seqs, 1, -1, 1), x, torch.zeros((), device=DEV)) for x in (k, v))
    last = torch.full((seqs, q_max), -1, device=DEV)  # the last key that a token sees
    last[seq, j] = place.long()
    seen = (key <= last.unsqueeze(2)) & held.unsqueeze(1)
    if c["window"]:
        seen &= (key > last.unsqueeze(2) - c["window"]) | (key < c["sinks"])
    score = (q @ k.transpose(2, 3) * s["scale"]).view(seqs, kv_heads, group, q_max, -1)
    score = score.masked_fill_(~seen.view(seqs, 1, 1, q_max, -1), -math.inf)
    top = score.amax(dim=4, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros((), device=DEV), top)
    p = score.sub_(top).exp_()
    total = p.sum(dim=4, keepdim=True)
    out = p.view(seqs, kv_heads, group * q_max, -1) @ v
    out = out.view(seqs, kv_heads, group, q_max, dim) / torch.where(total == 0, torch.ones((), device=DEV), total)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, q_max, heads, dim)[seq, j]
    result = {"out": out.to(DTYPES[c["dtype"]])}
    if s["lse"] is not None:
        lse = (top + total.log()).squeeze(4).permute(0, 3, 1, 2).reshape(seqs, q_max, heads)
        result["lse"] = lse[seq, j]
    return result


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append8" else _exact_attn(case, s)


def _exact_append(c, s):
    """The stored values before they are rounded to 8 bits, in units of their blocks' scales."""
    q_len, kv_len = _lengths(c)
    r, dim, block, page = c["rot"], c["dim"], c["block"], c["page"]
    places = torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(q_len, kv_len)]).double()
    turn = torch.tensor([1000000.0 ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device=DEV)
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(places, turn))

    def rotated(x, gamma):
        x = x.double()
        if gamma is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / dim + 1e-6) * gamma.double()
        pairs = [[2 * i, 2 * i + 1] if c["interleaved"] else [i, i + r // 2] for i in range(r // 2)]
        pairs = torch.tensor(pairs, device=DEV)
        w = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]]) * z[:, None, :]
        x = x.clone()
        x[..., pairs[:, 0]], x[..., pairs[:, 1]] = w.real, w.imag
        return x

    result = {"q": rotated(s["q"], s["gq"])}
    for name, x in (("k", rotated(s["k"], s["gk"])), ("v", s["v"].double())):
        codes = s[name + "_codes"].view(torch.float8_e4m3fn).double()
        scale = (s[name + "_scale"].double() - 127).exp2()
        at = 0
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            for start in range((m - n) // block * block, m, block):
                lo, hi = max(start, m - n), min(start + block, m)
                where, slot = int(s["table"][b, start // page]), start % page
                new = x[at + lo - (m - n):at + hi - (m - n)].transpose(0, 1)  # [head][token][dim]
                ratio = new.abs().amax((1, 2)) / LARGEST
                e = torch.where(ratio > 0, torch.ceil(torch.log2(ratio)), torch.full_like(ratio, LOWEST))
                e = e.clamp(LOWEST, HIGHEST).exp2()
                if lo > start:
                    was = scale[where, :, slot // block]
                    e = torch.maximum(e, was)
                    codes[where, :, slot:slot + lo - start] *= (was / e)[:, None, None]
                codes[where, :, slot + lo - start:slot + hi - start] = new / e[:, None, None]
                scale[where, :, slot // block] = e
            at += n
        result[name + "_codes"], result[name + "_scale"] = codes, scale
    return result


def _exact_attn(c, s):
    q_len, kv_len = _lengths(c)
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)

    def values(name, pages, h, m):
        if c["op"] == "window":
            return s[name + "_cache"][pages, h].reshape(-1, c["dim"])[:m].double()
        x = s[name + "_codes"][pages, h].view(torch.float8_e4m3fn).double().reshape(-1, c["dim"])
        e = s[name + "_scale"][pages, h].double().reshape(-1) - 127
        return (x * torch.repeat_interleave(e.exp2(), c["block"])[:, None])[:m]

    at = 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        pages = s["table"][b, :-(-m // c["page"])].long()
        place = torch.arange(m - n, m, device=DEV)[:, None]
        key = torch.arange(m, device=DEV)[None, :]
        hide = key > place
        if c["window"]:
            hide = hide | ((place - key >= c["window"]) & (key >= c["sinks"]))
        for h in range(c["kv_heads"]):
            k, v = values("k", pages, h, m), values("v", pages, h, m)
            for i in range(h * group, (h + 1) * group):
                w = (s["q"][at:at + n, i].double() @ k.t()).mul_(s["scale"]).masked_fill_(hide, -math.inf)
                total = torch.logsumexp(w, dim=1)
                lse[at:at + n, i] = total
                w = torch.nan_to_num(w.sub_(total[:, None]).exp_(), nan=0.0)  # rows that see nothing
                out[at:at + n, i] = w @ v
        at += n
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}
