"""The attention half of a layer on the GPU: paged attention, rotary append and the 4-bit
linear against 64-bit references, with error bounds derived from the arithmetic
(tests/attn_ref.py), at the sizes, masks and layouts where each can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import DT, FP32, HALF, attention, make_batch, q4_dense, rates, rotate  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()


class Dev:
    """A batch on the device: structs, workspace, outputs filled with a mark."""

    def __init__(self, bt, pad_rows=0, layout="heads", wide=0, max_q=None):
        self.bt = bt
        n = bt.tokens + pad_rows
        k, v = bt.k_cache.cuda(), bt.v_cache.cuda()
        if layout == "slots":  # [pages][slots][heads][dim] in memory
            k, v = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (k, v))
        if layout == "joint":  # k and v of a page next to each other
            both = torch.stack((k, v), 1)
            k, v = both[:, 0], both[:, 1]
        self.k, self.v = k, v
        q = torch.full((n, bt.heads * bt.dim + wide), 3.0, dtype=DT[bt.dtype], device="cuda")
        self.q = q[:, wide:].view(n, bt.heads, bt.dim)
        self.q[:bt.tokens] = bt.q.cuda()
        out = torch.full((n, bt.heads * bt.dim + wide), 7.0, dtype=DT[bt.dtype], device="cuda")
        self.out = out[:, :bt.heads * bt.dim].view(n, bt.heads, bt.dim)
        self.lse = torch.full((n, bt.heads), 7.0, device="cuda")
        self.shape = moe.make_attn_shape(n, len(bt.q_len), bt.heads, bt.kv_heads, bt.dim, bt.page, bt.pages,
                                         bt.table.shape[1], max(bt.q_len) if max_q is None else max_q, act=bt.dtype)
        self.cache = moe.make_kv_cache(self.k, self.v)
        self.kv_len = torch.tensor(bt.kv_len, dtype=torch.int32, device="cuda")
        self.table, self.cu_q = bt.table.cuda(), bt.cu_q.cuda()
        self.batch = moe.make_attn_batch(self.cu_q, self.kv_len, self.table)
        self.ws = torch.zeros(moe.moe_attn_workspace_size(self.shape), dtype=torch.uint8, device="cuda")

    def attend(self, scale, lse=True):
        moe.moe_paged_attention(self.shape, self.q, self.cache, self.batch, self.out, scale=scale,
                                lse=self.lse if lse else None, workspace=self.ws)
        torch.cuda.synchronize()
        return moe.moe_read_device_error(self.ws)


def check(bt, scale=None, **kw):
    d = Dev(bt, **kw)
    scale = bt.dim ** -0.5 if scale is None else scale
    assert d.attend(scale) == 0
    out, lse, tol, tol_lse = attention(bt, scale)
    got, got_lse = d.out[:bt.tokens].cpu().double(), d.lse[:bt.tokens].cpu().double()
    assert torch.isfinite(got).all()
    over = (got - out).abs() - tol
    assert (over <= 0).all(), f"off by {(got - out).abs().max()}, over the bound by {over.max()}"
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert (got[empty] == 0).all()
    assert ((got_lse - lse).abs()[~empty] <= tol_lse[~empty]).all()
    # padding rows stay as they were, and a second run (of a workspace in use) gives the same bits
    assert (d.out[bt.tokens:] == 7).all() and (d.lse[bt.tokens:] == 7).all()
    first, first_lse = d.out.clone(), d.lse.clone()
    assert d.attend(scale) == 0
    assert torch.equal(d.out, first) and torch.equal(d.lse, first_lse)
    return d


# name: dtype, heads, kv_heads, dim, page, chunk lengths, cache lengths
ATTN = {
    "one token one key": ("bf16", 8, 1, 128, 16, [1], [1]),
    "one token fp32": ("f32", 4, 4, 64, 16, [1], [3]),
    "decode ragged": ("bf16", 32, 4, 128, 16, [1] * 9, [1, 15, 16, 17, 100, 255, 256, 257, 700]),
    "decode no group": ("bf16", 5, 5, 128, 64, [1] * 3, [64, 65, 200]),
    "decode dim 64": ("bf16", 16, 2, 64, 32, [1] * 4, [31, 32, 33, 900]),
    "decode group 3": ("bf16", 12, 4, 128, 16, [1] * 5, [5, 77, 128, 300, 1025]),
    "decode group 16": ("bf16", 32, 2, 64, 128, [1] * 3, [129, 500, 40]),
    "decode group 20": ("bf16", 40, 2, 64, 16, [1, 1], [50, 333]),
    "decode many": ("bf16", 8, 2, 64, 16, [1] * 70, [1 + 13 * i % 190 for i in range(70)]),
    "decode long": ("bf16", 8, 1, 128, 64, [1], [9000]),
    "decode empty caches": ("bf16", 8, 2, 128, 16, [1, 1, 1, 1], [0, 40, 0, 1]),
    "idle sequences": ("bf16", 8, 2, 128, 16, [0, 1, 0, 1, 0], [20, 30, 0, 1, 7]),
    "decode 40 pairs": ("bf16", 16, 4, 128, 16, [1, 0, 1, 2, 1, 1, 1, 1, 1, 2], [700, 30, 0, 1, 1900, 65, 512, 513, 2, 40]),
    "decode 120 pairs": ("bf16", 24, 8, 64, 32, [1] * 15, [1 + 67 * i for i in range(15)]),
    "decode 200 pairs": ("bf16", 16, 8, 64, 16, [1, 2, 0, 1, 1] * 5, [(i * 41) % 500 for i in range(25)]),
    "decode 400 pairs": ("bf16", 8, 8, 128, 16, [1] * 50, [(i * 29) % 300 for i in range(50)]),
    "decode one pair long table": ("bf16", 16, 1, 64, 64, [1], [4096]),
    "few tokens": ("bf16", 8, 4, 128, 16, [3, 1, 5, 2], [3, 200, 97, 64]),
    "few tokens group 8": ("bf16", 16, 2, 64, 32, [2, 2, 1], [2, 100, 513]),
    "few tokens cut short": ("bf16", 8, 4, 128, 16, [4, 4, 4], [2, 0, 4]),
    "odd pages": ("bf16", 8, 2, 128, 5, [1, 1, 3], [11, 64, 100]),
    "page of one": ("bf16", 4, 2, 64, 1, [1, 2], [40, 5]),
    "odd head size": ("bf16", 6, 2, 72, 16, [1, 9], [40, 77]),
    "head size 8": ("f32", 3, 1, 8, 16, [4, 1], [40, 9]),
    "head size 256": ("bf16", 4, 2, 256, 16, [1, 17], [300, 60]),
    "head size 256 fp32": ("f32", 4, 2, 256, 12, [2, 17], [300, 60]),
    "chunk alone": ("bf16", 8, 1, 128, 64, [300], [300]),
    "chunk over cache": ("bf16", 8, 2, 128, 16, [129], [1000]),
    "chunk no group": ("bf16", 3, 3, 128, 32, [257], [400]),
    "chunk dim 64": ("bf16", 16, 2, 64, 32, [200, 33], [200, 500]),
    "chunk group 3": ("bf16", 6, 2, 128, 128, [100, 45], [400, 45]),
    "chunk group 5 odd": ("bf16", 5, 1, 64, 16, [77, 1, 30], [77, 130, 31]),
    "chunk ragged": ("bf16", 16, 4, 128, 16, [1, 64, 0, 130, 17], [500, 64, 9, 131, 700]),
    "chunk cut short": ("bf16", 8, 1, 128, 16, [150, 40], [40, 0]),
    "chunk page 256": ("bf16", 8, 2, 128, 256, [70, 140], [70, 700]),
    "chunk fp32": ("f32", 6, 2, 128, 16, [70, 1, 33], [70, 300, 64]),
    "chunk odd page": ("bf16", 8, 2, 128, 24, [100], [220]),
    "chunk tile ends": ("bf16", 8, 1, 128, 128, [16, 17, 32, 15], [128, 129, 256, 127]),
    "chunk many": ("bf16", 8, 2, 64, 16, [(i * 37) % 90 for i in range(40)], [(i * 37) % 90 + (i * 53) % 300 for i in range(40)]),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_attention(name):
    check(make_batch(*ATTN[name], seed=len(name)))


@pytest.mark.parametrize("seqs", [1, 6, 14, 34, 70, 90])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,most", [(8, 5), (32, 2), (60, 1), (4, 16)])
def test_attention_rows_of_a_pair(seqs, dim, heads, most):
    # up to 16 query rows a key head, for every number of CTAs that a pair can get
    q_len = [most - i % 2 if most > 1 else 1 for i in range(seqs)]
    check(make_batch("bf16", heads, 4, dim, 32, q_len, [q_len[i] + (i * 19) % 44 for i in range(seqs)], seed=seqs))


@pytest.mark.parametrize("name", ["decode ragged", "few tokens", "chunk ragged", "chunk fp32"])
@pytest.mark.parametrize("layout", ["slots", "joint"])
def test_attention_layouts(name, layout):
    # other cache layouts, q and out as slices of wider rows, padding rows, a loose max_q
    bt = make_batch(*ATTN[name], seed=3)
    check(bt, layout=layout, wide=64, pad_rows=5, max_q=min(bt.tokens, max(bt.q_len) + 2))


@pytest.mark.parametrize("name", ["decode ragged", "few tokens", "chunk ragged", "chunk over cache"])
@pytest.mark.parametrize("spread,scale", [(12.0, None), (1.0, 0.0), (1.0, -0.3)])
def test_attention_peaked_flat_and_negative(name, spread, scale):
    # one key takes nearly everything; every key the same; a negative factor
    check(make_batch(*ATTN[name], seed=8, spread=spread), scale=scale)


@pytest.mark.parametrize("fill", [math.inf, -math.inf])
@pytest.mark.parametrize("name", ["decode ragged", "chunk ragged", "odd pages"])
def test_attention_unwritten_slots(name, fill):
    check(make_batch(*ATTN[name], seed=4, fill=fill))


@pytest.mark.parametrize("name", ["decode ragged", "chunk ragged", "chunk fp32"])
def test_attention_rising_scores(name):
    # each key scores higher than all before it: the running maximum moves in every tile
    bt = make_batch(*ATTN[name], seed=5)
    bt.q[:] = 1.0
    for b, m in enumerate(bt.kv_len):
        p = torch.arange(m)
        level = (p.double() / 50).to(DT[bt.dtype])
        bt.k_cache[bt.table[b, p // bt.page].long(), :, p % bt.page] = level[:, None, None]
    check(bt, scale=40.0 / bt.dim)


@pytest.mark.parametrize("name", ["decode ragged", "chunk over cache", "odd pages"])
def test_attention_bad_data_is_recorded(name):
    # a page that does not exist, a chunk past max_q, a cache length past the table: recorded,
    # and every other sequence is right
    bt = make_batch(*ATTN[name], seed=6)
    spec = list(ATTN[name])
    spec[5], spec[6] = bt.q_len + [bt.q_len[0]], bt.kv_len + [70]
    spec[6][-1] = max(70, spec[5][-1])
    bt = make_batch(*spec, seed=6, fill=0.0)
    out, _, tol, _ = attention(bt, 0.1)
    good = int(bt.cu_q[-2])
    for what in ("page high", "page low", "cache length"):
        d = Dev(bt)
        if what == "page high":
            d.table[-1, 0] = bt.pages
        elif what == "page low":
            d.table[-1, 1] = -1
        else:
            d.kv_len[-1] = bt.table.shape[1] * bt.page + 1
            d.table[-1] = 0
        assert d.attend(0.1) == -7
        assert ((d.out.cpu().double() - out).abs() <= tol)[:good].all()
        assert moe.moe_read_device_error(d.ws) == 0  # read and cleared


@pytest.mark.parametrize("name", ["decode ragged", "chunk over cache", "chunk ragged", "odd pages"])
@pytest.mark.parametrize("what", ["falls", "leaves", "negative"])
def test_attention_bad_rows_are_recorded(name, what):
    # a cu_q that falls or leaves the rows: recorded, nothing outside the arrays is touched, and the
    # next call with the right one is right
    bt = make_batch(*ATTN[name], seed=12)
    d = Dev(bt, pad_rows=2)
    good = d.cu_q.clone()
    if what == "falls":
        d.cu_q[-1] = -5 if len(bt.q_len) == 1 else int(good[-2]) - 1
    elif what == "leaves":
        d.cu_q[-1] = bt.tokens + 1000
    else:
        d.cu_q[0] = -1000
    assert d.attend(0.1) == -7
    d.cu_q.copy_(good)
    d.out.fill_(7.0)
    assert d.attend(0.1) == 0
    out, _, tol, _ = attention(bt, 0.1)
    assert ((d.out[:bt.tokens].cpu().double() - out).abs() <= tol).all() and (d.out[bt.tokens:] == 7).all()


def test_attention_graph_and_streams():
    # replays of a captured graph see new lengths and new data; two streams with their own
    # workspaces do not disturb each other
    bts = [make_batch(*ATTN["decode ragged"], seed=s) for s in (1, 2)]
    d = Dev(bts[0])
    side = torch.cuda.Stream()
    d.attend(0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        moe.moe_paged_attention(d.shape, d.q, d.cache, d.batch, d.out, scale=0.1, lse=d.lse, workspace=d.ws)
    for bt in bts:
        d.q.copy_(bt.q)
        d.k.copy_(bt.k_cache)
        d.v.copy_(bt.v_cache)
        d.table.copy_(bt.table)
        kv = [max(1, n // 2) for n in bt.kv_len] if bt is bts[1] else bt.kv_len
        d.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        bt.kv_len = kv
        g.replay()
        torch.cuda.synchronize()
        out, _, tol, _ = attention(bt, 0.1)
        assert ((d.out.cpu().double() - out).abs() <= tol).all()
    a, b = (Dev(make_batch(*ATTN[n], seed=9)) for n in ("decode ragged", "chunk ragged"))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st in ((a, s1), (b, s2)):
            moe.moe_paged_attention(x.shape, x.q, x.cache, x.batch, x.out, scale=0.1, workspace=x.ws, stream=st)
    torch.cuda.synchronize()
    for x in (a, b):
        out, _, tol, _ = attention(x.bt, 0.1)
        assert ((x.out.cpu().double() - out).abs() <= tol).all()


def test_attention_wait_that_runs_out():
    # the softmax arrivals of the chunk kernel can never be enough: the wait ends after its limit
    # with an error recorded, and the next ordinary call is right
    bt = make_batch(*ATTN["chunk over cache"], seed=7)
    d = Dev(bt)
    moe.moe_debug_set_waits(1_000_000, 1)
    try:
        assert d.attend(0.1) == -7
    finally:
        moe.moe_debug_set_waits()
    assert d.attend(0.1) == 0
    out, _, tol, _ = attention(bt, 0.1)
    assert ((d.out.cpu().double() - out).abs() <= tol).all()


@pytest.mark.parametrize("q_len", [1, 40])
def test_attention_far_pages(q_len):
    # element offsets past 2^32 in the cache: the pages of a small batch lie at its far end
    bt = make_batch("bf16", 8, 2, 128, 64, [q_len], [300], seed=11)
    n = (1 << 32) // (2 * 64 * 128) + 8
    d = Dev(bt)
    big = torch.empty(n, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    at = n - bt.pages
    big[at:] = d.k
    vbig = torch.empty_like(big)
    vbig[at:] = d.v
    d.shape.n_pages = n
    d.cache = moe.make_kv_cache(big, vbig)
    used = -(-300 // 64)
    d.table[:, :used] += at
    assert d.attend(0.1) == 0
    out, _, tol, _ = attention(bt, 0.1)
    assert ((d.out.cpu().double() - out).abs() <= tol).all()


# ------------------------------------------------------------------------------- rotary append

ROPE = {
    # dtype, heads, kv_heads, dim, page, chunks, caches, rot, interleaved, norm, scaling, factor, offset
    "decode": ("bf16", 32, 4, 128, 16, [1] * 8, [1, 5, 16, 17, 100, 64, 33, 2], 128, False, True, "none", 1.0, None),
    "prompt yarn": ("bf16", 8, 2, 128, 64, [70, 1, 130], [70, 9, 200], 128, False, True, "yarn", 4.0, 100000),
    "interleaved part": ("f32", 6, 3, 96, 24, [33, 5], [40, 5], 64, True, False, "ntk", 8.0, 900000),
    "half part": ("f32", 4, 1, 80, 10, [7, 20], [9, 33], 32, False, True, "linear", 4.0, None),
    "smallest": ("bf16", 1, 1, 16, 1, [1], [1], 16, True, False, "none", 1.0, None),
    "widest": ("bf16", 3, 1, 256, 16, [5, 0, 3], [5, 2, 50], 256, False, True, "none", 1.0, 2**31 - 100),
    "widest interleaved": ("f32", 3, 3, 256, 7, [5, 3], [5, 50], 240, True, True, "none", 1.0, None),
    "cut short": ("bf16", 8, 2, 64, 16, [6, 4], [2, 0], 64, False, False, "none", 1.0, 50),
    "negative positions": ("f32", 2, 2, 32, 16, [6], [9], 32, False, False, "none", 1.0, -20),
    "many tokens": ("bf16", 5, 1, 64, 16, [1, 900, 0, 2047], [4, 900, 3, 2100], 32, False, True, "none", 1.0, None),
    "many tokens fp32": ("f32", 3, 1, 24, 3, [1300, 1, 1200], [1300, 1, 1201], 16, True, False, "none", 1.0, 7),
    "many sequences": ("bf16", 4, 2, 64, 16, [i % 3 for i in range(600)], [i % 3 + i % 7 for i in range(600)], 64, True,
                       False, "none", 1.0, None),
}


def _rope_case(name, in_place=False, layout="heads", pad=3):
    dt, heads, kvh, dim, page, ql, kl, rot, inter, norm, scaling, factor, offset = ROPE[name]
    g = torch.Generator().manual_seed(len(name))
    bt = make_batch(dt, heads, kvh, dim, page, ql, kl, seed=2, fill=5.0)
    n = bt.tokens
    qkv = torch.randn(n + pad, (heads + 2 * kvh) * dim, generator=g).to(DT[dt])
    gq, gk = ((1 + 0.2 * torch.randn(dim, generator=g)).to(DT[dt]) if norm else None for _ in range(2))
    place = torch.cat([torch.arange(m - c, m) for c, m in zip(ql, kl)]) if n else torch.zeros(0)
    pos = place if offset is None else place + offset
    dev = qkv.cuda()
    q, k, v = dev.split([heads * dim, kvh * dim, kvh * dim], 1)
    q, k, v = q.view(-1, heads, dim), k.view(-1, kvh, dim), v.view(-1, kvh, dim)
    d = Dev(bt, pad_rows=pad, layout=layout)
    q_out = q if in_place else d.out
    rope = moe.make_rope(rot, base=1e6, interleaved=inter, scaling=scaling, factor=factor, trained_len=32768,
                         q_gamma=None if gq is None else gq.cuda(), k_gamma=None if gk is None else gk.cuda())
    positions = None if offset is None else torch.nn.functional.pad(pos, (0, pad)).int().cuda()
    moe.moe_rope_append(d.shape, rope, q, k, v, d.cache, d.batch, q_out, positions=positions, workspace=d.ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(d.ws) == 0
    f, ms = rates(rot, 1e6, scaling, factor, 32768)
    hq, hk, hv = qkv[:n].split([heads * dim, kvh * dim, kvh * dim], 1)
    want_q = rotate(hq.view(n, heads, dim), pos, f, ms, inter, gq)
    want_k = rotate(hk.view(n, kvh, dim), pos, f, ms, inter, gk)
    k_cache, v_cache, k_tol = bt.k_cache.double(), bt.v_cache.double(), torch.zeros(bt.k_cache.shape).double()

    def bound(want, x, gamma):
        # a rotated pair is off by the cosine and sine (2^-22 with the angle's rounding), three
        # products and sums, and a norm's dim additions, relative to the pair's size before
        size = rotate(x, torch.zeros(n), [0.0] * (rot // 2), ms, inter, gamma).abs().amax(-1, keepdim=True)
        return (8 * FP32 + (dim * FP32 if gamma is not None else 0)) * 2 * size + HALF[dt] * want.abs()

    q_tol, kk_tol = bound(want_q, hq.view(n, heads, dim), gq), bound(want_k, hk.view(n, kvh, dim), gk)
    at = 0
    for b, (c, m) in enumerate(zip(ql, kl)):
        for j in range(c):
            p = m - c + j
            if p >= 0:
                pg = int(bt.table[b, p // page])
                k_cache[pg, :, p % page], v_cache[pg, :, p % page] = want_k[at], hv.view(n, kvh, dim)[at].double()
                k_tol[pg, :, p % page] = kk_tol[at]
            at += 1
    got_q = q_out.cpu().double()
    assert ((got_q[:n] - want_q).abs() <= q_tol).all(), ((got_q[:n] - want_q).abs() - q_tol).max()
    assert ((d.k.cpu().double() - k_cache).abs() <= k_tol).all()  # slots of no new token: unchanged
    assert torch.equal(d.v.cpu().double(), v_cache)
    if not in_place:
        assert (q_out[n:] == 7).all()


@pytest.mark.parametrize("name", list(ROPE))
def test_rope_append(name):
    _rope_case(name)


@pytest.mark.parametrize("name", ["decode", "prompt yarn", "interleaved part", "half part"])
@pytest.mark.parametrize("in_place,layout", [(True, "slots"), (False, "joint")])
def test_rope_append_in_place_and_layouts(name, in_place, layout):
    _rope_case(name, in_place, layout)


@pytest.mark.parametrize("cu", [[0, 9, 4], [0, 3, 5000], [-7, 3, 6]])
def test_rope_append_bad_rows_are_recorded(cu):
    bt = make_batch("bf16", 4, 2, 64, 16, [3, 3], [3, 20], seed=1, fill=5.0)
    d = Dev(bt)
    d.cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
    x = torch.randn(bt.tokens, 4, 64, device="cuda").bfloat16()
    moe.moe_rope_append(d.shape, moe.make_rope(64), x, x[:, :2].contiguous(), x[:, 2:].contiguous(), d.cache, d.batch,
                        d.out, workspace=d.ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(d.ws) == -7


def test_rope_append_bad_page_is_recorded_and_skipped():
    bt = make_batch("bf16", 4, 2, 64, 16, [3, 20], [3, 20], seed=1, fill=5.0)
    d = Dev(bt)
    x = torch.randn(bt.tokens, 4, 64, device="cuda").bfloat16()
    rope = moe.make_rope(64)
    for bad in (bt.pages, -1):
        d.table[1, 1] = bad
        before = d.k.clone()
        d.k.fill_(5.0)
        moe.moe_rope_append(d.shape, rope, x, x[:, :2].contiguous(), x[:, 2:].contiguous(), d.cache, d.batch, d.out,
                            workspace=d.ws)
        torch.cuda.synchronize()
        assert moe.moe_read_device_error(d.ws) == -7
        changed = (d.k != 5.0).any(-1).any(1)  # [pages][slots]
        assert int(changed.sum()) == 3 + 16  # the tokens of the good pages
        assert torch.isfinite(d.out).all()
        d.k.copy_(before)


# ------------------------------------------------------------------------------- 4-bit linear

UNIFORM = [-1 + 2 * j / 15 for j in range(16)]
NORMAL = [math.sqrt(2) * float(torch.erfinv(torch.tensor(2 * (j + 0.5) / 16 - 1, dtype=torch.float64))) for j in range(16)]
SHIFTED = [0.25 * (j - 3) for j in range(16)]


@pytest.mark.parametrize("book", [UNIFORM, NORMAL, SHIFTED], ids=["uniform", "normal", "shifted"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,q_block", [
    (1, 64, 1, 64), (1, 2048, 640, 64), (8, 512, 129, 64), (3, 96, 17, 32), (7, 4064, 515, 32), (16, 1024, 256, 128),
    (17, 768, 100, 64), (33, 640, 65, 128), (64, 2048, 200, 64), (65, 256, 48, 32), (130, 512, 33, 64), (2, 8, 5, 2),
    (20, 2112, 4100, 64), (70, 4224, 2050, 128), (33, 512, 140000, 64), (9, 8192, 1030, 64), (64, 8192, 1100, 256),
    (20, 192, 40000, 64), (3, 320, 20001, 64), (40, 96, 19999, 32), (11, 4160, 130, 64), (16, 8192, 300, 512),
    (5, 240, 31, 48), (9, 176, 40, 16), (4, 8192, 24, 256), (1, 5632, 2047, 128), (12, 32, 64, 32)])
def test_q4_linear(T, K, N, q_block, out, book):
    g = torch.Generator().manual_seed(T * 1000 + K + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    scales = (torch.rand(N, K // q_block, generator=g) + 0.25).bfloat16()
    x = torch.randn(T, K + 16, generator=g).bfloat16()
    res = torch.randn(T, N + 3, generator=g).bfloat16()
    w = q4_dense(codes, scales, [float(torch.tensor(b).float()) for b in book], q_block)
    want = x[:, 8:K + 8].double() @ w.T
    size = x[:, 8:K + 8].double().abs() @ w.abs().T
    shape = moe.make_q4_linear_shape(T, K, N, out, q_block)
    weight = moe.make_q4_weight(codes.cuda(), scales.cuda(), book)
    xd, rd = x.cuda()[:, 8:K + 8], res.cuda()
    for with_res in (False, True):
        buf = torch.full((T, N + 5), 7.0, dtype=DT[out], device="cuda")
        moe.moe_q4_linear(shape, xd, weight, buf[:, :N], residual=rd[:, :N] if with_res else None)
        torch.cuda.synchronize()
        ref = want + res[:, :N].double() if with_res else want
        # K products and sums in fp32 in some order (each at most one step of the sizes' sum), a
        # codebook value held to 2^-17, one rounding of the result
        tol = size * (min(K, 512) + K / 64 + 16) * FP32 + size * 2.0 ** -17 + (HALF[out] + FP32) * ref.abs() + 1e-30
        got = buf[:, :N].cpu().double()
        assert ((got - ref).abs() <= tol).all(), ((got - ref).abs() - tol).max()
        assert (buf[:, N:] == 7).all()
        again = torch.empty_like(buf)
        moe.moe_q4_linear(shape, xd, weight, again[:, :N], residual=rd[:, :N] if with_res else None)
        assert torch.equal(again[:, :N], buf[:, :N])


def test_q4_linear_wait_that_runs_out():
    # the tensor-core kernel's operands can never be complete: the wait ends after its limit with an
    # error recorded, and the next ordinary call is right
    g = torch.Generator().manual_seed(2)
    codes = torch.randint(0, 256, (4100, 1024), generator=g).to(torch.uint8)
    scales = (torch.rand(4100, 32, generator=g) + 0.25).bfloat16()
    x = torch.randn(20, 2048, generator=g).bfloat16()
    shape, weight = moe.make_q4_linear_shape(20, 2048, 4100, "f32"), moe.make_q4_weight(codes.cuda(), scales.cuda(), UNIFORM)
    out = torch.empty(20, 4100, device="cuda")
    moe.moe_debug_set_waits(1_000_000, 1)
    try:
        moe.moe_q4_linear(shape, x.cuda(), weight, out)
        assert moe.moe_q4_linear_read_error() == -7
    finally:
        moe.moe_debug_set_waits()
    moe.moe_q4_linear(shape, x.cuda(), weight, out)
    assert moe.moe_q4_linear_read_error() == 0
    want = x.double() @ q4_dense(codes, scales, UNIFORM, 64).T
    assert (out.cpu().double() - want).abs().max() <= 2e-3


def test_q4_linear_residual_in_place():
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (96, 128), generator=g).to(torch.uint8).cuda()
    scales = (torch.rand(96, 4, generator=g) + 0.25).bfloat16().cuda()
    x, res = (torch.randn(5, n, generator=g).bfloat16().cuda() for n in (256, 96))
    shape, weight = moe.make_q4_linear_shape(5, 256, 96), moe.make_q4_weight(codes, scales, UNIFORM)
    a, b = torch.empty_like(res), res.clone()
    moe.moe_q4_linear(shape, x, weight, a, residual=res)
    moe.moe_q4_linear(shape, x, weight, b, residual=b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,K,N,q_block", [(7, 512, 300, 64), (16, 192, 2000, 32), (33, 640, 40000, 64), (40, 96, 70, 32)])
def test_q4_linear_keeps_fp32_values(T, K, N, q_block):
    # rows of x with a single one: each result is one weight, codebook value times scale.  Its value is
    # held to 24 bits (three roundings of its parts' sum), the product with the scale rounds once more;
    # the start of the sum and the empty blocks add zeros.
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    scales = (torch.rand(N, K // q_block, generator=g) + 0.25).bfloat16()
    x = torch.zeros(T, K)
    x[torch.arange(T), torch.randperm(K, generator=g)[:T]] = 1.0
    book = [float(torch.tensor(b).float()) for b in NORMAL]
    want = x.double() @ q4_dense(codes, scales, book, q_block).T
    shape, weight = moe.make_q4_linear_shape(T, K, N, "f32", q_block), moe.make_q4_weight(codes.cuda(), scales.cuda(), NORMAL)
    out = torch.empty(T, N, device="cuda")
    moe.moe_q4_linear(shape, x.bfloat16().cuda(), weight, out)
    assert ((out.cpu().double() - want).abs() <= 6 * FP32 * want.abs()).all()
