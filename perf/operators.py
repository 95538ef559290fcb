"""The attention half of a decoder layer next to the MoE block: what is measured, and its plain form.

Three operators that a serving step runs one after another: rotary positions with the write
into a paged key/value cache ("rope"), attention of chunks of new tokens over that cache
("attn"), and the products with 4-bit weights that surround them ("q4").
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 8 sequences: the smallest call, latency only
        dict(name="rope decode", op="rope", dtype="bf16", seqs=8, q_min=1, q_max=1, past=900, heads=32, kv_heads=4,
             dim=128, rot=128, interleaved=False, norm=True, scaling="none", factor=1.0, offset=0, page=16, lens=1),
        # prompts of 3 requests prefilled in one call, positions scaled for a long context
        dict(name="rope prompt", op="rope", dtype="bf16", seqs=3, q_min=1100, q_max=1700, past=0, heads=32,
             kv_heads=4, dim=128, rot=128, interleaved=False, norm=True, scaling="yarn", factor=4.0, offset=40000,
             page=64, lens=2),
        # fp32, interleaved pairs on part of an odd head size, far positions, pages that are no power of two
        dict(name="rope part fp32", op="rope", dtype="f32", seqs=5, q_min=101, q_max=411, past=37, heads=12,
             kv_heads=3, dim=96, rot=64, interleaved=True, norm=False, scaling="ntk", factor=8.0, offset=250000,
             page=24, lens=3),
        # one decode step of 8 sequences at short contexts
        dict(name="attn decode short", op="attn", dtype="bf16", seqs=8, q_min=1, q_max=1, kv_min=90, kv_max=1100,
             heads=32, kv_heads=4, dim=128, page=16, lse=False, short=False, lens=4),
        # a full decode batch, ragged contexts of up to 16k tokens
        dict(name="attn decode batch", op="attn", dtype="bf16", seqs=64, q_min=1, q_max=1, kv_min=500, kv_max=16000,
             heads=32, kv_heads=4, dim=128, page=64, lse=False, short=False, lens=5),
        # a single user at a very long context: the split over the cache decides
        dict(name="attn decode long", op="attn", dtype="bf16", seqs=1, q_min=1, q_max=1, kv_min=131071, kv_max=131071,
             heads=32, kv_heads=4, dim=128, page=128, lse=True, short=False, lens=6),
        # a few tokens each (draft tokens to be checked), fp32, odd group, head and page sizes
        dict(name="attn few fp32", op="attn", dtype="f32", seqs=6, q_min=1, q_max=5, kv_min=3, kv_max=1500,
             heads=12, kv_heads=4, dim=80, page=10, lse=True, short=False, lens=7),
        # a chunk of a long prompt over what is already cached: the largest call
        dict(name="attn chunk", op="attn", dtype="bf16", seqs=1, q_min=2048, q_max=2048, kv_min=16384, kv_max=16384,
             heads=32, kv_heads=4, dim=128, page=64, lse=False, short=False, lens=8),
        # a mixed step: chunks and single tokens, one sequence whose first rows see no key
        dict(name="attn mixed", op="attn", dtype="bf16", seqs=7, q_min=1, q_max=900, kv_min=5, kv_max=5000,
             heads=16, kv_heads=2, dim=64, page=32, lse=True, short=True, lens=9),
        # the qkv projection of a single token
        dict(name="q4 one token", op="q4", rows=1, k=2048, n=5120, group=64, book="uniform", residual=False,
             out="bf16"),
        # a general codebook, small groups, odd sizes, with the residual
        dict(name="q4 odd", op="q4", rows=7, k=4064, n=2047, group=32, book="normal", residual=True, out="bf16"),
        # the vocabulary product of a decode batch, fp32 logits
        dict(name="q4 vocabulary", op="q4", rows=16, k=2048, n=131072, group=64, book="uniform", residual=False,
             out="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        sizes = [v for v in c.values() if type(v) is int]
        if w["bytes"] <= 1.0e9 and w["flops"] <= 2.5e11 and 3072 not in sizes:
            return c


def _draw(rng):
    op = rng.choice(["rope", "attn", "attn", "q4"])
    if op == "q4":
        group = rng.choice([32, 64, 64, 128])
        return dict(op="q4", rows=_log(rng, 1, 64), k=group * _log(rng, 512 // group, 8192 // group),
                    n=_log(rng, 100, 30000), group=group, book=rng.choice(["uniform", "uniform", "normal"]),
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
    common = dict(heads=heads, kv_heads=kv_heads, lens=rng.randrange(1 << 30))
    if op == "rope":
        dim = rng.choice([64, 96, 128, 128, 256])
        q_max = rng.choice([1, _log(rng, 2, 1500)])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op="rope", dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=_log(rng, 1, 12) if q_max > 1 else
                    _log(rng, 1, 64), q_min=1, q_max=q_max, past=rng.randrange(200), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.5,
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    offset=_log(rng, 1, 500000), page=rng.choice([1, 16, 24, 64, 128]), **common)
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
    return dict(op="attn", dtype=dtype, seqs=seqs, q_min=1, q_max=q_max, kv_min=max(1, kv_max // 20), kv_max=kv_max,
                dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), lse=rng.random() < 0.5,
                short=q_max > 1 and rng.random() < 0.25, **common)


# ------------------------------------------------------------------------------- inputs

def _lengths(c):
    """The chunk and cache lengths of the case's sequences: lists, the same for every seed."""
    r = random.Random(c["lens"])
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["seqs"])]
    q[r.randrange(c["seqs"])] = c["q_max"]
    if c["op"] == "rope":
        return q, [n + r.randint(0, c["past"]) for n in q]
    kv = [r.randint(c["kv_min"], c["kv_max"]) for _ in range(c["seqs"])]
    kv[r.randrange(c["seqs"])] = c["kv_max"]
    kv = [max(n, m) for n, m in zip(q, kv)]  # a sequence's keys include its chunk's own
    if c["short"]:  # but for one, cut short: its first rows see no key
        i = r.randrange(c["seqs"])
        kv[i] = max(1, q[i] // 2)
    return q, kv


def _pairs(q, kv):
    """How many (token, key) pairs the causal rule lets through."""
    total = 0
    for n, m in zip(q, kv):
        first = max(0, n - m)  # tokens that see no key
        total += sum((m - n + first + 1, m)) * (n - first) // 2
    return total


def work(case):
    c = case
    if c["op"] == "q4":
        t, k, n = c["rows"], c["k"], c["n"]
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": n * k // 2 + n * (k // c["group"]) * 2 + t * k * 2 + t * n * (size + 2 * c["residual"]),
                "flops": 2 * t * k * n}
    q, kv = _lengths(c)
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        values = sum(q) * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * values * size, "flops": 6 * values}
    seen = sum(kv)
    rows = sum(q) * c["heads"]
    return {"bytes": 2 * rows * c["dim"] * size + 2 * seen * c["kv_heads"] * c["dim"] * size + 4 * rows * c["lse"],
            "flops": 4 * _pairs(q, kv) * c["heads"] * c["dim"]}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _frequencies(c):
    """The rotation rates (radians a position) of the pairs of one head in 64 bits, and the factor on the rotated
    part: plain, all slowed down (linear), a larger base (ntk), or slow pairs only (yarn)."""
    r, base, factor, trained = c["rot"], 1000000.0, c["factor"], 32768
    if c["scaling"] == "ntk":
        base = base * factor ** (r / (r - 2))
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    f = torch.pow(torch.tensor(base, dtype=torch.float64, device=DEV), -2 * i / r)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "yarn":
        turns = lambda n: r * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), r - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


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


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] == "q4":
        t, k, n = c["rows"], c["k"], c["n"]
        s["x"] = torch.randn(t, k, generator=g, device=DEV).bfloat16()
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = ((torch.rand(n, k // c["group"], generator=g, device=DEV) + 0.5) * 2 / math.sqrt(k)).bfloat16()
        book = [-1 + 2 * j / 15 for j in range(16)]
        if c["book"] == "normal":  # quantiles of a normal distribution, a common choice for trained weights
            z = [math.sqrt(2) * torch.erfinv(torch.tensor(2 * (j + 0.5) / 16 - 1, dtype=torch.float64)).item()
                 for j in range(16)]
            book = [v / z[15] for v in z]
        s["book"] = torch.tensor(book, dtype=torch.float32, device=DEV)
        s["residual"] = torch.randn(t, n, generator=g, device=DEV).bfloat16() if c["residual"] else None
        s["out"] = torch.empty(t, n, dtype=DTYPES[c["out"]], device=DEV)
        if own:
            import top_routing_grouped_router_gb300 as moe
            s["shape"] = moe.make_q4_linear_shape(t, k, n, out=c["out"], q_block=c["group"])
            s["weight"] = moe.make_q4_weight(s["codes"], s["scales"], book)
        return s

    q_len, kv_len = _lengths(c)
    n, dt = sum(q_len), DTYPES[c["dtype"]]
    heads, kv_heads, dim = c["heads"], c["kv_heads"], c["dim"]
    s["table"], pages = _paging(c, kv_len, g)
    s["cu_q"] = torch.tensor([0] + q_len, device=DEV).cumsum(0).int()
    s["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device=DEV)
    s["q_max"], s["tokens"] = max(q_len), n
    cache = (pages, kv_heads, c["page"], dim)
    if c["op"] == "rope":
        # q, k and v are slices of the projection's output
        qkv = torch.randn(n, (heads + 2 * kv_heads) * dim, generator=g, device=DEV).to(dt)
        q, k, v = qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], dim=1)
        s["q"], s["k"], s["v"] = q.view(n, heads, dim), k.view(n, kv_heads, dim), v.view(n, kv_heads, dim)
        s["k_cache"], s["v_cache"] = (torch.zeros(cache, dtype=dt, device=DEV) for _ in range(2))
        s["q_out"] = torch.empty(n, heads, dim, dtype=dt, device=DEV)
        s["gq"], s["gk"] = ((1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(dt) if c["norm"] else None
                            for _ in range(2))
        ends = torch.repeat_interleave(s["cu_q"][1:], torch.tensor(q_len, device=DEV))
        last = torch.repeat_interleave(s["kv_len"], torch.tensor(q_len, device=DEV))
        s["positions"] = (torch.arange(n, device=DEV) - ends + last + c["offset"]).int()
        s["rates"], s["factor"] = _frequencies(c)
    else:
        # scores with a spread of about 1.5, as trained heads have; what no sequence has written is NaN
        s["q"] = (1.5 * torch.randn(n, heads, dim, generator=g, device=DEV)).to(dt)
        s["k_cache"] = torch.randn(cache, generator=g, device=DEV, dtype=torch.float32).to(dt)
        s["v_cache"] = torch.randn(cache, generator=g, device=DEV, dtype=torch.float32).to(dt)
        slot = torch.arange(s["table"].shape[1] * c["page"], device=DEV).view(1, -1, c["page"])
        used = torch.zeros(pages, c["page"], dtype=torch.bool, device=DEV)
        held = s["table"] >= 0
        used[s["table"][held].long()] = (slot < s["kv_len"].view(-1, 1, 1))[held]
        for name in ("k_cache", "v_cache"):
            s[name].masked_fill_(~used.view(pages, 1, c["page"], 1), float("nan"))
        s["out"] = torch.empty(n, heads, dim, dtype=dt, device=DEV)
        s["lse"] = torch.empty(n, heads, dtype=torch.float32, device=DEV) if c["lse"] else None
        s["scale"] = 1 / math.sqrt(dim)
    if own:
        import top_routing_grouped_router_gb300 as moe
        s["shape"] = moe.make_attn_shape(n, c["seqs"], heads, kv_heads, dim, c["page"], pages, s["table"].shape[1],
                                         s["q_max"], act=c["dtype"])
        s["cache"] = moe.make_kv_cache(s["k_cache"], s["v_cache"])
        s["batch"] = moe.make_attn_batch(s["cu_q"], s["kv_len"], s["table"])
        s["ws"] = torch.zeros(moe.moe_attn_workspace_size(s["shape"]), dtype=torch.uint8, device=DEV)
        if c["op"] == "rope":
            s["rope"] = moe.make_rope(c["rot"], base=1000000.0, interleaved=c["interleaved"], scaling=c["scaling"],
                                      factor=c["factor"], trained_len=32768, q_gamma=s["gq"], k_gamma=s["gk"],
                                      eps=1e-6)
    return s


# ------------------------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import top_routing_grouped_router_gb300 as moe
        if op == "q4":
            moe.moe_q4_linear(s["shape"], s["x"], s["weight"], s["out"], residual=s["residual"])
            return s["out"]
        if op == "rope":
            moe.moe_rope_append(s["shape"], s["rope"], s["q"], s["k"], s["v"], s["cache"], s["batch"], s["q_out"],
                                positions=s["positions"], workspace=s["ws"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        moe.moe_paged_attention(s["shape"], s["q"], s["cache"], s["batch"], s["out"], scale=s["scale"], lse=s["lse"],
                                workspace=s["ws"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    return {"q4": _plain_q4, "rope": _plain_rope, "attn": _plain_attn}[op](s)


def _plain_q4(s):
    c = s["c"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=2).view(c["n"], c["k"])  # low nibble first
    w = s["book"][codes.int()].view(c["n"], -1, c["group"]) * s["scales"].float().unsqueeze(2)
    y = s["x"].float() @ w.view(c["n"], c["k"]).t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _rows_of(s):
    """For each new token its sequence and its place in the sequence."""
    at = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(s["cu_q"], at.int(), right=True) - 1
    place = s["kv_len"][seq] - (s["cu_q"][seq + 1] - at)
    return seq, place


def _norm(x, gamma):
    return x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * gamma.float()


def _plain_rope(s):
    c = s["c"]
    angle = s["positions"].double().unsqueeze(1) * s["rates"]
    cos, sin = ((s["factor"] * f(angle)).float().unsqueeze(1) for f in (torch.cos, torch.sin))

    def turn(x, gamma):
        x = x.float()
        if gamma is not None:
            x = _norm(x, gamma)
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=3).flatten(2)
        else:
            a, b = r.chunk(2, dim=2)
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=2)
        return torch.cat((r, rest), dim=2)

    dt = DTYPES[c["dtype"]]
    seq, place = _rows_of(s)
    page = s["table"][seq, place // c["page"]].long()
    slot = place % c["page"]
    s["k_cache"][page, :, slot] = turn(s["k"], s["gk"]).to(dt)
    s["v_cache"][page, :, slot] = s["v"]
    return {"q": turn(s["q"], s["gq"]).to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
    k, v = (s[name][table].permute(0, 2, 1, 3, 4).reshape(seqs, kv_heads, -1, dim).float()
            for name in ("k_cache", "v_cache"))
    key = torch.arange(k.shape[2], device=DEV)
    held = key < s["kv_len"].unsqueeze(1)
    k, v = (torch.where(held.view(seqs, 1, -1, 1), x, torch.zeros((), device=DEV)) for x in (k, v))
    last = torch.full((seqs, q_max), -1, device=DEV)  # the last key that a token sees
    last[seq, j] = place.long()
    seen = (key <= last.unsqueeze(2)) & held.unsqueeze(1)
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
    return {"q4": _exact_q4, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](case, s)


def _exact_q4(c, s):
    x, book = s["x"].double(), s["book"].double()
    y = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device=DEV)
    for half, shift in ((0, 0), (1, 4)):  # the even elements of a row are in the low nibbles, the odd in the high
        w = book[((s["codes"] >> shift) & 15).long()]
        w = w * s["scales"].double().repeat_interleave(c["group"] // 2, dim=1)
        y += torch.einsum("nk,tk->tn", w, x[:, half::2])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rope(c, s):
    q_len, kv_len = _lengths(c)
    r, dim = c["rot"], c["dim"]
    base, factor, size = 1000000.0, c["factor"], 1.0
    if c["scaling"] == "ntk":
        base *= factor ** (r / (r - 2.0))
    rates = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        rates = [f / factor for f in rates]
    if c["scaling"] == "yarn":
        size = 1 + 0.1 * math.log(factor)
        edge = [r * math.log(32768 / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32, 1)]
        low, high = max(0, math.floor(edge[0])), min(r - 1, math.ceil(edge[1]))
        for i in range(r // 2):
            part = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            rates[i] = rates[i] * ((1 - part) + part / factor)
    turn = torch.tensor(rates, dtype=torch.float64, device=DEV)
    z = torch.polar(torch.full((sum(q_len), r // 2), size, dtype=torch.float64, device=DEV),
                    torch.outer(s["positions"].double(), turn))

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

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k, v, at = rotated(s["k"], s["gk"]), s["v"].double(), 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        place = torch.arange(m - n, m, device=DEV)
        page = s["table"][b][torch.div(place, c["page"], rounding_mode="floor")].long()
        k_cache[page, :, place % c["page"]] = k[at:at + n]
        v_cache[page, :, place % c["page"]] = v[at:at + n]
        at += n
    return {"q": rotated(s["q"], s["gq"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attn(c, s):
    q_len, kv_len = _lengths(c)
    group = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        pages = s["table"][b, :-(-m // c["page"])].long()
        hide = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        for h in range(c["kv_heads"]):
            k, v = (s[x][pages, h].reshape(-1, c["dim"])[:m].double() for x in ("k_cache", "v_cache"))
            for i in range(h * group, (h + 1) * group):
                w = (s["q"][at:at + n, i].double() @ k.t()).mul_(s["scale"]).masked_fill_(hide, -math.inf)
                total = torch.logsumexp(w, dim=1)
                lse[at:at + n, i] = total
                w = torch.nan_to_num(w.sub_(total[:, None]).exp_(), nan=0.0)  # rows that see nothing
                out[at:at + n, i] = w @ v
        at += n
    return {"out": out} if s["lse"] is None else {"out": out, "lse": lse}
