"""The 8-bit paged cache and attention with a window on the GPU, against 64-bit references with bounds derived
from the arithmetic (tests/q8_ref.py), at the sizes, masks and layouts where they can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import DT, FP32, make_batch, rates, rotate  # noqa: E402
from q8_ref import HIGHEST, LARGEST, LOWEST, attention, exponents, from_codes, power, round8, step8, store  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()


def laid_out(x, layout):
    """x [pages][heads][slots][...] with the same values in another order in memory."""
    x = x.cuda()
    return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "slots" else x


class Dev:
    """A batch on the device, over its own cache (block None) or an 8-bit one with a scale for `block` tokens."""

    def __init__(self, bt, block=None, pad_rows=0, layout="heads", wide=0, max_q=None):
        self.bt, self.block = bt, block
        n = bt.tokens + pad_rows
        q = torch.full((n, bt.heads * bt.dim + wide), 3.0, dtype=DT[bt.dtype], device="cuda")
        self.q = q[:, wide:].view(n, bt.heads, bt.dim)
        self.q[:bt.tokens] = bt.q.cuda()
        out = torch.full((n, bt.heads * bt.dim + wide), 7.0, dtype=DT[bt.dtype], device="cuda")
        self.out = out[:, :bt.heads * bt.dim].view(n, bt.heads, bt.dim)
        self.lse = torch.full((n, bt.heads), 7.0, device="cuda")
        self.shape = moe.make_attn_shape(n, len(bt.q_len), bt.heads, bt.kv_heads, bt.dim, bt.page, bt.pages,
                                         bt.table.shape[1], max(bt.q_len) if max_q is None else max_q, act=bt.dtype)
        self.kv_len = torch.tensor(bt.kv_len, dtype=torch.int32, device="cuda")
        self.table, self.cu_q = bt.table.cuda(), bt.cu_q.cuda()
        self.batch = moe.make_attn_batch(self.cu_q, self.kv_len, self.table)
        if block is None:
            self.k, self.v = (laid_out(c, layout) for c in (bt.k_cache, bt.v_cache))
            self.cache, size = moe.make_kv_cache(self.k, self.v), moe.moe_attn_workspace_size(self.shape)
        else:  # the batch's values are from now on those that the codes stand for
            (k, self.ks, bt.k_cache), (v, self.vs, bt.v_cache) = store(bt.k_cache, block), store(bt.v_cache, block)
            self.k, self.v = laid_out(k, layout), laid_out(v, layout)
            self.ks, self.vs = laid_out(self.ks, "heads"), laid_out(self.vs, "heads")
            if layout == "slots":  # a scale's heads in rows of their own, padded
                wide_s = [torch.zeros(*s.shape[:2], s.shape[2] + 3, dtype=torch.uint8, device="cuda") for s in (self.ks, self.vs)]
                for w, s in zip(wide_s, (self.ks, self.vs)):
                    w[..., :s.shape[2]] = s
                self.ks, self.vs = (w[..., :s.shape[2]] for w, s in zip(wide_s, (self.ks, self.vs)))
            self.cache = moe.make_kv_cache_q8(self.k, self.v, self.ks, self.vs)
            size = moe.moe_attn_q8_workspace_size(self.shape, block)
        self.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def attend(self, scale, window=None, sinks=0, lse=True, stream=None):
        w = None if window is None else moe.make_attn_window(window, sinks)
        kw = dict(scale=scale, lse=self.lse if lse else None, workspace=self.ws, stream=stream)
        if self.block is not None:
            moe.moe_paged_attention_q8(self.shape, self.q, self.cache, self.batch, self.out, window=w, **kw)
        else:
            moe.moe_paged_attention_window(self.shape, self.q, self.cache, self.batch, w, self.out, **kw)

    def errors(self):
        torch.cuda.synchronize()
        return moe.moe_read_device_error(self.ws)


def check(bt, block=None, window=None, sinks=0, scale=None, **kw):
    d = Dev(bt, block, **kw)
    scale = bt.dim ** -0.5 if scale is None else scale
    d.attend(scale, window, sinks)
    assert d.errors() == 0
    out, lse, tol, tol_lse = attention(bt, scale, window, sinks)
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
    d.attend(scale, window, sinks)
    assert d.errors() == 0
    assert torch.equal(d.out, first) and torch.equal(d.lse, first_lse)
    return d


# name: dtype, heads, kv_heads, dim, page, chunk lengths, cache lengths
BATCH = {
    "one token one key": ("bf16", 8, 1, 128, 16, [1], [1]),
    "one token fp32": ("f32", 4, 4, 64, 16, [1], [3]),
    "decode ragged": ("bf16", 32, 4, 128, 16, [1] * 9, [1, 15, 16, 17, 100, 255, 256, 257, 700]),
    "decode no group": ("bf16", 5, 5, 128, 64, [1] * 3, [64, 65, 200]),
    "decode dim 64": ("bf16", 16, 2, 64, 32, [1] * 4, [31, 32, 33, 900]),
    "decode group 3": ("bf16", 12, 4, 128, 16, [1] * 5, [5, 77, 128, 300, 1025]),
    "decode group 16": ("bf16", 32, 2, 64, 128, [1] * 3, [129, 500, 40]),
    "decode group 20": ("bf16", 40, 2, 64, 16, [1, 1], [50, 333]),
    "decode many": ("bf16", 8, 2, 64, 16, [1] * 70, [1 + 13 * i % 190 for i in range(70)]),
    "decode line 200": ("bf16", 4, 1, 128, 16, [1 + i % 4 for i in range(200)], [5 + (i * 53) % 700 for i in range(200)]),
    "decode long": ("bf16", 8, 1, 128, 64, [1], [9000]),
    "decode empty caches": ("bf16", 8, 2, 128, 16, [1, 1, 1, 1], [0, 40, 0, 1]),
    "idle sequences": ("bf16", 8, 2, 128, 16, [0, 1, 0, 1, 0], [20, 30, 0, 1, 7]),
    "few tokens": ("bf16", 8, 4, 128, 16, [3, 1, 5, 2], [3, 200, 97, 64]),
    "few tokens cut short": ("bf16", 8, 4, 128, 16, [4, 4, 4], [2, 0, 4]),
    "odd head size": ("bf16", 6, 2, 80, 16, [1, 9], [40, 77]),
    "odd pages": ("bf16", 8, 2, 128, 24, [1, 1, 3], [11, 64, 100]),
    "head size 16": ("f32", 3, 1, 16, 16, [4, 1], [40, 9]),
    "head size 256": ("bf16", 4, 2, 256, 16, [1, 17], [300, 60]),
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
    "chunk many": ("bf16", 8, 2, 64, 16, [(i * 37) % 90 for i in range(40)], [(i * 37) % 90 + (i * 53) % 300 for i in range(40)]),
    "chunk many long": ("bf16", 4, 1, 128, 16, [(i * 37) % 90 for i in range(40)], [(i * 37) % 90 + (i * 153) % 900 for i in range(40)]),
}
# windows shorter than a group of keys and longer than the caches, on and beside the borders of steps; first keys
# from none to more than a step
WINDOWS = [(1, 0), (1, 3), (7, 0), (16, 16), (17, 1), (127, 5), (128, 0), (129, 130), (300, 4), (2**31 - 1, 0), (5, 2**31 - 1)]


@pytest.mark.parametrize("name", list(BATCH))
def test_window(name):
    for i, (window, sinks) in enumerate(WINDOWS):
        check(make_batch(*BATCH[name], seed=i), window=window, sinks=sinks)


@pytest.mark.parametrize("name", list(BATCH))
@pytest.mark.parametrize("blocks", ["page", 16, 1])
def test_q8(name, blocks):
    spec = BATCH[name]
    block = spec[4] if blocks == "page" else math.gcd(blocks, spec[4])
    check(make_batch(*spec, seed=len(name)), block=block)


@pytest.mark.parametrize("name", list(BATCH))
def test_q8_window(name):
    for i, (window, sinks) in enumerate(WINDOWS):
        check(make_batch(*BATCH[name], seed=20 + i), block=math.gcd(16, BATCH[name][4]), window=window, sinks=sinks)


LAYOUTS = ["decode ragged", "few tokens", "chunk ragged", "chunk fp32"]


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("block", [None, 16, 8])
def test_layouts(name, block):
    # another order of the cache, q and out as slices of wider rows, padding rows, a loose max_q
    bt = make_batch(*BATCH[name], seed=3)
    check(bt, block=block, window=90, sinks=2, layout="slots", wide=64, pad_rows=5,
          max_q=min(bt.tokens, max(bt.q_len) + 2))


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("spread,scale", [(12.0, None), (1.0, 0.0), (1.0, -0.3)])
def test_peaked_flat_and_negative(name, spread, scale):
    check(make_batch(*BATCH[name], seed=8, spread=spread), window=50, sinks=3, scale=scale)
    check(make_batch(*BATCH[name], seed=8, spread=spread), block=16, scale=scale)


@pytest.mark.parametrize("name", ["decode ragged", "few tokens", "chunk ragged", "chunk over cache", "chunk dim 64", "chunk fp32"])
def test_q8_scales_that_differ_widely(name):
    # blocks of keys and of values in very different sizes; queries far from 1, of each head its own
    bt = make_batch(*BATCH[name], seed=9)
    g = torch.Generator().manual_seed(1)
    for c, most in ((bt.k_cache, 3), (bt.v_cache, 12)):
        e = torch.randint(-most, most + 1, (*c.shape[:2], c.shape[2] // 16, 1, 1), generator=g).double()
        c.copy_((c.double().unflatten(2, (-1, 16)) * e.exp2()).flatten(2, 3))
    bt.q *= (torch.arange(bt.heads) * 4.0 - 30).exp2()[:, None].to(bt.q.dtype)
    check(bt, block=16)


@pytest.mark.parametrize("name", ["few tokens", "chunk alone", "chunk over cache", "chunk dim 64", "chunk fp32"])
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("power_of", [8, 18, 26])
def test_q8_a_large_block_that_few_tokens_see(name, what, power_of):
    # the last tokens' keys or values are far larger than all before: those who do not see them get what they see as
    # exactly as ever, and those who do what dominates
    bt = make_batch(*BATCH[name], seed=19)
    for b, m in enumerate(bt.kv_len):
        page, slot = int(bt.table[b, (m - 1) // bt.page]), (m - 1) % bt.page // 16 * 16
        for c in (bt.k_cache,) * (what != "v") + (bt.v_cache,) * (what != "k"):
            c[page, :, slot:slot + 16] = (c[page, :, slot:slot + 16].double() * 2.0 ** power_of).to(c.dtype)
    if what == "k":
        bt.q *= 0.125
    check(bt, block=16)


@pytest.mark.parametrize("name", ["decode ragged", "chunk ragged", "odd pages", "chunk fp32"])
@pytest.mark.parametrize("block", [None, 8])
def test_what_no_token_sees_is_not_read(name, block):
    # table entries of pages outside the window are wrong, slots outside it hold NaN
    window, sinks = 40, 3
    bt = make_batch(*BATCH[name], seed=4)
    d = Dev(bt, block)
    out, lse, tol, _ = attention(bt, 0.1, window, sinks)
    for b, (n, m) in enumerate(zip(bt.q_len, bt.kv_len)):
        p = torch.arange(m)
        first = max(0, m - n) - window + 1 if n else m  # the first key of the first token's window
        hidden = (p < first) & (p >= sinks)
        for pi in range(-(-m // bt.page)):
            on = slice(pi * bt.page, min(m, (pi + 1) * bt.page))
            page = int(bt.table[b, pi])
            slots = torch.nonzero(hidden[on])[:, 0].cuda()
            for c in (d.k, d.v):
                c[page, :, slots] = math.nan if block is None else 0x7f
            if hidden[on].all():
                d.table[b, pi] = 1 << 30
    d.attend(0.1, window, sinks)
    assert d.errors() == 0
    assert ((d.out.cpu().double() - out).abs() <= tol).all()
    assert torch.equal(d.lse.cpu() == -math.inf, lse == -math.inf)


@pytest.mark.parametrize("name", ["decode ragged", "few tokens", "chunk over cache", "chunk dim 64", "chunk fp32"])
@pytest.mark.parametrize("what", ["query", "key", "value", "key scale", "value scale"])
def test_q8_nan_reaches_those_who_see_it(name, what):
    # the key or value of the last new token of a sequence, of head 0: its last row sees it
    bt = make_batch(*BATCH[name], seed=13)
    b = max(range(len(bt.q_len)), key=lambda i: bt.q_len[i] * 10000 + bt.kv_len[i])
    t, p, group = int(bt.cu_q[b + 1]) - 1, bt.kv_len[b] - 1, bt.heads // bt.kv_heads
    page, slot = int(bt.table[b, p // bt.page]), p % bt.page
    d = Dev(bt, 16)
    out, _, tol, _ = attention(bt, 0.1)
    if what == "query":
        d.q[t, :group] = math.nan
    elif what in ("key", "value"):
        (d.k if what == "key" else d.v)[page, 0, slot, 5] = 0xff
    else:
        (d.ks if "key" in what else d.vs)[page, 0, slot // 16] = 255
    d.attend(0.1)
    assert d.errors() == 0
    got = d.out.cpu().double()
    assert got[t, :group].isnan().any(-1).all()
    others = torch.ones(bt.tokens, bt.heads, dtype=torch.bool)
    others[int(bt.cu_q[b]):t + 1, :group] = False
    assert ((got - out).abs() <= tol)[others].all()


@pytest.mark.parametrize("name", ["decode ragged", "chunk over cache", "odd pages"])
@pytest.mark.parametrize("block", [None, 8])
def test_wrong_data_is_recorded(name, block):
    # a page that does not exist, a cache length past the table, a cu_q that leaves the rows
    bt = make_batch(*BATCH[name], seed=6, fill=0.0)
    for what in ("page high", "page low", "cache length", "rows"):
        d = Dev(bt, block)
        if what == "page high":
            d.table[-1, 0] = bt.pages
        elif what == "page low":
            d.table[-1, 0] = -1
        elif what == "cache length":
            d.kv_len[-1] = bt.table.shape[1] * bt.page + 1
            d.table[-1] = 0
        else:
            d.cu_q[-1] = bt.tokens + 1000
        d.attend(0.1, 10**6, 1)
        assert d.errors() == -7 and d.errors() == 0


@pytest.mark.parametrize("name", ["decode ragged", "chunk ragged"])
@pytest.mark.parametrize("block", [None, 16])
def test_graph_and_streams(name, block):
    # replays of a captured graph see new lengths and data; two streams with their own workspaces
    bt = make_batch(*BATCH[name], seed=1)
    d, e = Dev(bt, block), Dev(make_batch(*BATCH[name], seed=2), block)
    want = attention(bt, 0.1, 60, 4)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    d.attend(0.1, 60, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        d.attend(0.1, 60, 4, stream=side)
    for i in range(3):
        d.out.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(10):
            g.replay()
            e.attend(0.1, 60, 4, stream=other)
        assert d.errors() == 0 and e.errors() == 0
        assert ((d.out.cpu().double() - want[0]).abs() <= want[2]).all()
        got = attention(e.bt, 0.1, 60, 4)
        assert ((e.out.cpu().double() - got[0]).abs() <= got[2]).all()
        kv = [max(n, m - 7 * (i + 1)) for n, m in zip(bt.q_len, bt.kv_len)]
        bt.kv_len = kv
        d.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        want = attention(bt, 0.1, 60, 4)


@pytest.mark.parametrize("q_len", [1, 40])
def test_q8_far_pages(q_len):
    # byte offsets past 2^32 in the cache: the pages of a small batch lie at its far end
    bt = make_batch("bf16", 8, 2, 128, 64, [q_len], [300], seed=11)
    d = Dev(bt, 32)
    n = (1 << 32) // (2 * 64 * 128) + 8
    at = n - bt.pages
    big = []
    for c in (d.k, d.v):
        big.append(torch.empty(n, 2, 64, 128, dtype=torch.uint8, device="cuda"))
        big[-1][at:] = c
    scales = []
    for c in (d.ks, d.vs):
        scales.append(torch.empty(n, 2, 2, dtype=torch.uint8, device="cuda"))
        scales[-1][at:] = c
    d.shape.n_pages = n
    d.cache = moe.make_kv_cache_q8(*big, *scales)
    d.table[:, :-(-300 // 64)] += at
    d.attend(0.1)
    assert d.errors() == 0
    out, _, tol, _ = attention(bt, 0.1)
    assert ((d.out.cpu().double() - out).abs() <= tol).all()


@pytest.mark.parametrize("name", ["decode ragged", "decode line 200", "few tokens cut short", "chunk ragged", "chunk cut short", "chunk dim 64",
                                  "odd pages"])
@pytest.mark.parametrize("block,window", [(None, 60), (16, 60), (16, None), (8, 60)])
def test_without_the_sums_the_outputs_are_the_same(name, block, window):
    bt = make_batch(*BATCH[name], seed=5)
    d = Dev(bt, math.gcd(block, bt.page) if block else None)
    d.attend(0.1, window, 4)
    torch.cuda.synchronize()
    first = d.out.clone()
    d.out.fill_(7.0)
    d.lse.fill_(7.0)
    d.attend(0.1, window, 4, lse=False)
    assert d.errors() == 0
    assert torch.equal(d.out, first) and (d.lse == 7).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block,window", [(None, 20), (16, 20), (16, None)])
@pytest.mark.parametrize("longest", [60, 900])
def test_more_sequences_than_a_scan_and_a_list_hold(dim, block, window, longest):
    # rounds of 128, 384 and 512 sequences; up to 512 keys no item is cut, and a CTA has dozens of them
    ql = [(i * 7) % 4 for i in range(1300)]
    kl = [n + (i * 13) % 50 for i, n in enumerate(ql)]
    ql[700], kl[700], ql[1299], kl[1299] = 40, 50, 21, longest
    check(make_batch("bf16", 8, 4, dim, 16, ql, kl, seed=6), block, window, 3)


@pytest.mark.parametrize("block", [None, 16])
def test_graphs_of_different_kernels_share_a_workspace(block):
    # one after another on a stream: what one leaves in the workspace does not disturb the next
    names = ["decode line 200", "chunk over cache", "decode ragged", "chunk many long", "head size 16", "chunk dim 64"]
    runs = [Dev(make_batch(*BATCH[n], seed=i), block) for i, n in enumerate(names)]
    ws = torch.zeros(max(d.ws.numel() for d in runs), dtype=torch.uint8, device="cuda")
    graphs, first, side = [], [], torch.cuda.Stream()
    for d in runs:
        d.attend(0.1, 200, 4)
        assert d.errors() == 0
        first.append((d.out.clone(), d.lse.clone()))
        d.ws = ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            d.attend(0.1, 200, 4, stream=side)
        graphs.append(g)
    for order in ([0, 1, 2, 3, 4, 5], [5, 3, 1, 0, 2, 4], [1, 1, 0, 0, 3, 2, 5, 4]):
        for d in runs:
            d.out.fill_(7.0)
            d.lse.fill_(7.0)
        for i in order:
            graphs[i].replay()
        assert runs[0].errors() == 0
        for d, (out, lse) in zip(runs, first):
            assert torch.equal(d.out, out) and torch.equal(d.lse, lse)


@pytest.mark.parametrize("q_len", [1, 30])
@pytest.mark.parametrize("block,window", [(None, 40), (16, None)])
def test_a_page_that_a_sequence_lists_twice(q_len, block, window):
    bt = make_batch("bf16", 8, 2, 64, 16, [q_len], [96], seed=3)
    bt.table[0, 3] = bt.table[0, 1]
    bt.table[0, 4] = bt.table[0, 1]
    check(bt, block, window, 2)


FEW_PAIRS = {
    # up to eight (sequence, key head) pairs with many keys: heads, kv_heads, dim, page, chunk lengths, cache lengths
    "one pair": (8, 1, 128, 16, [1], [5003]),
    "one pair dim 64": (5, 1, 64, 64, [3], [2000]),
    "wide group": (32, 2, 128, 16, [1], [3001]),
    "four pairs": (16, 2, 128, 32, [1, 2], [2500, 1900]),
    "most empty": (8, 1, 64, 16, [1, 0, 1, 2], [4000, 70, 5, 1]),
    "eight pairs": (32, 4, 128, 16, [1, 2], [6000, 4001]),
    "cut short": (8, 4, 64, 16, [4], [2]),
}


@pytest.mark.parametrize("name", list(FEW_PAIRS))
@pytest.mark.parametrize("block", [None, 16, 32])
@pytest.mark.parametrize("window,sinks", [(None, 0), (700, 3), (1500, 900), (3300, 0), (600, 0)])
def test_few_pairs_with_many_keys(name, block, window, sinks):
    heads, kvh, dim, page, ql, kl = FEW_PAIRS[name]
    if block is not None and page % block or block is None and window is None:
        pytest.skip("no such case")
    bt = make_batch("bf16", heads, kvh, dim, page, ql, kl, seed=12)
    if name == "cut short":  # a table for many more keys
        bt.table = torch.nn.functional.pad(bt.table, (0, 200), value=-7)
    d = check(bt, block, window, sinks)
    first = d.out.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for _ in range(3):  # the next begins while the one before ends
            d.attend(dim ** -0.5, window, sinks, stream=side)
    d.out.fill_(7.0)
    g.replay()
    assert d.errors() == 0
    assert torch.equal(d.out, first)


@pytest.mark.parametrize("ql,kl", [([1, 1, 1], [100, 90, 70]), ([40, 25, 30], [100, 90, 94])])
@pytest.mark.parametrize("block,window", [(None, 50), (16, None), (8, 50)])
def test_sequences_that_share_pages(ql, kl, block, window):
    bt = make_batch("bf16", 8, 2, 128, 16, ql, kl, seed=8)
    bt.table[1, :4] = bt.table[0, :4]  # whole pages of a common prefix
    bt.table[2] = bt.table[0]
    check(bt, block, window, 5)


# ------------------------------------------------------------------------------- rotary append

APPEND = {
    # dtype, heads, kv_heads, dim, page, block, chunks, caches, rot, interleaved, norm, offset of positions
    "decode": ("bf16", 32, 4, 128, 16, 16, [1] * 8, [1, 5, 16, 17, 100, 64, 33, 2], 128, False, True, None),
    "decode page scales": ("bf16", 8, 2, 128, 64, 64, [1] * 5, [1, 63, 64, 65, 100], 128, False, False, None),
    "decode token scales": ("bf16", 8, 2, 64, 16, 1, [1] * 5, [1, 63, 64, 65, 100], 64, True, False, 1000),
    "prompt": ("bf16", 8, 2, 128, 64, 64, [70, 1, 130], [70, 9, 200], 128, False, True, 100000),
    "prompt small blocks": ("bf16", 8, 2, 128, 64, 8, [70, 1, 130], [75, 9, 201], 128, False, True, None),
    "prompt blocks of 128": ("bf16", 6, 3, 128, 256, 128, [300, 5], [333, 130], 64, True, False, None),
    "prompt blocks of 256": ("bf16", 4, 1, 128, 256, 256, [600, 100], [633, 130], 128, False, True, None),
    "interleaved part": ("f32", 6, 3, 96, 24, 24, [33, 5], [40, 5], 64, True, False, 900000),
    "half part": ("f32", 4, 1, 80, 10, 5, [7, 20], [9, 33], 32, False, True, None),
    "smallest": ("bf16", 1, 1, 16, 1, 1, [1], [1], 16, True, False, None),
    "heads of 32": ("bf16", 2, 1, 32, 48, 48, [50, 3], [60, 40], 32, False, True, None),
    "widest": ("bf16", 3, 1, 256, 16, 16, [5, 0, 3], [5, 2, 50], 256, False, True, 2**31 - 100),
    "widest long": ("f32", 3, 3, 256, 128, 128, [200, 3], [207, 50], 240, True, True, None),
    "cut short": ("bf16", 8, 2, 64, 16, 16, [6, 4], [2, 0], 64, False, False, 50),
    "negative positions": ("f32", 2, 2, 32, 16, 16, [6], [9], 32, False, False, -20),
    "many tokens": ("bf16", 5, 1, 64, 16, 16, [1, 900, 0, 2047], [4, 900, 3, 2100], 32, False, True, None),
    "many sequences": ("bf16", 4, 2, 64, 16, 16, [i % 3 for i in range(600)], [i % 3 + i % 7 for i in range(600)], 64, True,
                       False, None),
}


class Append:
    """A case's inputs on the host and the device; `run` appends, `check` compares the cache with the definition."""

    def __init__(self, spec, seed=0, layout="heads", pad=3, spread=1.0):
        (dt, self.heads, self.kvh, self.dim, self.page, self.block, self.ql, self.kl, self.rot, self.inter, norm,
         offset) = spec
        g = torch.Generator().manual_seed(seed)
        bt = make_batch(dt, self.heads, self.kvh, self.dim, self.page, self.ql, self.kl, seed=2, fill=1.5)
        self.bt, n = bt, bt.tokens
        self.d = Dev(bt, self.block, pad_rows=pad, layout=layout)
        qkv = (spread * torch.randn(n + pad, (self.heads + 2 * self.kvh) * self.dim, generator=g)).to(DT[dt])
        self.gq, self.gk = ((1 + 0.2 * torch.randn(self.dim, generator=g)).to(DT[dt]) if norm else None for _ in range(2))
        place = torch.cat([torch.arange(m - c, m) for c, m in zip(self.ql, self.kl)])
        self.place, self.pos = place, place if offset is None else place + offset
        self.positions = None if offset is None else torch.nn.functional.pad(self.pos, (0, pad)).int().cuda()
        self.rope = moe.make_rope(self.rot, base=1e6, interleaved=self.inter, q_gamma=None if self.gq is None else self.gq.cuda(),
                                  k_gamma=None if self.gk is None else self.gk.cuda())
        self.set(qkv)

    def set(self, qkv):
        self.qkv, dev, n = qkv, qkv.cuda(), self.bt.tokens
        q, k, v = dev.split([self.heads * self.dim, self.kvh * self.dim, self.kvh * self.dim], 1)
        self.q, self.k, self.v = (x.view(len(qkv), -1, self.dim) for x in (q, k, v))
        hq, hk, hv = (x.view(n, -1, self.dim) for x in qkv[:n].split([self.heads * self.dim, self.kvh * self.dim,
                                                                    self.kvh * self.dim], 1))
        f, ms = rates(self.rot, 1e6)
        self.want_q, self.want_k = (rotate(x, self.pos, f, ms, self.inter, gamma) for x, gamma in ((hq, self.gq), (hk, self.gk)))
        self.want_v = hv.double()
        # a value is off by a few roundings in the norm (a sum of dim squares) and the rotation, relative to its pair
        self.err = (self.dim + 24) * FP32

    def run(self, q_out=None, stream=None):
        moe.moe_rope_append_q8(self.d.shape, self.rope, self.q, self.k, self.v, self.d.cache, self.d.batch,
                               self.d.out if q_out is None else q_out, positions=self.positions, workspace=self.d.ws,
                               stream=stream)

    def state(self):
        return [x.clone().cpu() for x in (self.d.k, self.d.ks, self.d.v, self.d.vs)]

    def check(self, before):
        """Every slot of the cache against what `before` and the new tokens make of it."""
        after = self.state()
        for i, (want, exact) in enumerate(((self.want_k, False), (self.want_v, True))):
            codes0, s0, codes1, s1 = before[2 * i], before[2 * i + 1].int() - 127, after[2 * i], after[2 * i + 1].int() - 127
            values0 = from_codes(codes0.contiguous()) * power(s0).repeat_interleave(self.block, 2)[..., None]
            seen = torch.zeros(codes0.shape[0], codes0.shape[2], dtype=torch.bool)  # slots that were looked at
            blocks = torch.zeros(s0.shape[0], s0.shape[2], dtype=torch.bool)
            at = 0
            for b, (n, m) in enumerate(zip(self.ql, self.kl)):
                first = max(m - n, 0)
                for start in range(first // self.block * self.block, m if n else 0, self.block):
                    lo, hi = max(start, first), min(start + self.block, m)
                    page, slot = int(self.bt.table[b, start // self.page]), start % self.page
                    y = want[at + lo - (m - n):at + hi - (m - n)].transpose(0, 1)  # [head][token][dim]
                    old = slice(slot, slot + lo - start)
                    new = slice(slot + lo - start, slot + hi - start)
                    top = torch.where(y.isfinite(), y.abs(), torch.zeros(())).amax((1, 2))
                    e = s1[page, :, slot // self.block]
                    err = 0.0 if exact else self.err
                    was = s0[page, :, slot // self.block] if lo > start else torch.full_like(e, LOWEST)
                    assert (e >= torch.maximum(exponents(top * (1 - err)), was)).all()
                    assert (e <= torch.maximum(exponents(top * (1 + err)), was)).all()
                    s = power(e)[:, None, None]
                    got = from_codes(codes1[page, :, new].contiguous())
                    assert torch.equal(got.isnan(), ~y.isfinite())
                    t = (y / s).nan_to_num(nan=0.0, posinf=0.0, neginf=0.0).clamp(-LARGEST, LARGEST)
                    got = got.nan_to_num(nan=0.0)
                    if exact:
                        assert torch.equal(got, round8(t))
                    else:  # half a step, and what the value before rounding is off by, of its pair's size
                        size = (t.abs() + err * t.abs().amax()) * err + err * t.abs().amax()
                        assert ((got - t).abs() <= torch.maximum(step8(t), step8(got)) / 2 + size).all()
                    moved = values0[page, :, old] / s
                    kept = from_codes(codes1[page, :, old].contiguous())
                    assert torch.equal(kept, round8(moved))  # unmoved ones are what they were
                    seen[page, old.start:new.stop] = True
                    blocks[page, slot // self.block] = True
                at += n
            # everything else stays as it was, the bytes of untouched blocks among it
            same = (codes0 == codes1).all(3).all(1) | seen
            assert same.all()
            assert ((s0 == s1).all(1) | blocks).all()


@pytest.mark.parametrize("name", list(APPEND))
@pytest.mark.parametrize("layout", ["heads", "slots"])
def test_append(name, layout):
    a = Append(APPEND[name], seed=len(name), layout=layout)
    before = a.state()
    a.run()
    assert a.d.errors() == 0
    a.check(before)
    got, n = a.d.out.cpu(), a.bt.tokens
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[a.bt.dtype]
    size = a.want_q.abs().amax(2, keepdim=True)
    assert ((got[:n].double() - a.want_q).abs() <= half * a.want_q.abs() + (1 + half) * a.err * size).all()
    assert (got[n:] == 7).all()
    # the same again changes nothing
    after, out = a.state(), a.d.out.clone()
    a.run()
    assert a.d.errors() == 0
    assert all(torch.equal(x, y) for x, y in zip(after, a.state())) and torch.equal(out, a.d.out)


@pytest.mark.parametrize("name", ["decode", "decode page scales", "prompt small blocks", "interleaved part"])
@pytest.mark.parametrize("spread", [2.0 ** -9, 2.0 ** 5, 2.0 ** 30, 0.0])
def test_append_beside_older_tokens(name, spread):
    # new values far smaller and far larger than what the block holds, and zeros
    a = Append(APPEND[name], seed=5, spread=spread)
    before = a.state()
    a.run()
    assert a.d.errors() == 0
    a.check(before)


def test_append_of_the_largest_and_smallest_values():
    spec = ("f32", 2, 2, 64, 16, 16, [20, 3], [20, 30], 64, False, False, None)
    for value in (3.0e38, 1e-36, 1e-44, 448.0 * 2.0 ** 20, 448.0 * 2.0 ** 20 * (1 + 2.0 ** -23)):
        a = Append(spec, seed=1)
        qkv = torch.zeros_like(a.qkv)
        qkv[:, 4 * 64::5] = value  # v only: no rotation
        qkv[1:, 4 * 64::7] = -value / 3
        a.set(qkv)
        before = a.state()
        a.run()
        assert a.d.errors() == 0
        a.check(before)
        assert a.state()[3].max() <= HIGHEST + 127


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_append_of_values_that_are_not_finite(bad):
    a = Append(APPEND["prompt"], seed=3)
    qkv = a.qkv.clone()
    qkv[3, -5] = bad  # of v
    qkv[40, -a.dim:] = bad
    a.set(qkv)
    before = a.state()
    a.run()
    assert a.d.errors() == 0
    a.check(before)


def test_append_in_place_and_in_a_graph():
    a = Append(APPEND["decode"], seed=7)
    a.run()
    assert a.d.errors() == 0
    out, first = a.d.out.clone(), a.state()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        a.run(stream=side)
    a.d.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a.d.out) and all(torch.equal(x, y) for x, y in zip(first, a.state()))
    q = a.q.clone()
    a.q = q
    a.run(q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q[:a.bt.tokens], out[:a.bt.tokens])


def test_append_to_far_pages():
    # byte offsets past 2^32 in the cache
    a = Append(APPEND["decode page scales"], seed=4)
    before, d = a.state(), a.d
    n = (1 << 32) // (2 * 64 * 128) + 8
    at = n - a.bt.pages
    big = [torch.empty(n, *c.shape[1:], dtype=torch.uint8, device="cuda") for c in (d.k, d.v, d.ks, d.vs)]
    for to, c in zip(big, (d.k, d.v, d.ks, d.vs)):
        to[at:] = c
    d.shape.n_pages = n
    d.cache = moe.make_kv_cache_q8(*big)
    d.table += at
    a.run()
    assert d.errors() == 0
    for to, c in zip((d.k, d.v, d.ks, d.vs), big):
        to.copy_(c[at:])
    a.check(before)


@pytest.mark.parametrize("what", ["negative length", "length past the table", "idle length past the table", "long chunk",
                                  "page"])
def test_append_records_wrong_data(what):
    # and stores what the other sequences bring all the same
    a = Append(("bf16", 4, 2, 64, 16, 16, [3, 0, 70, 2], [5, 9, 71, 4], 64, False, False, None), seed=1)
    before = a.state()
    a.run()
    assert a.d.errors() == 0
    right = a.state()
    for x, y in zip((a.d.k, a.d.ks, a.d.v, a.d.vs), before):
        x.copy_(y)
    if what == "negative length":
        a.d.kv_len[2] = -1
    elif what == "length past the table":
        a.d.kv_len[2] = a.bt.table.shape[1] * 16 + 1
    elif what == "idle length past the table":
        a.d.kv_len[1] = a.bt.table.shape[1] * 16 + 1
    elif what == "page":
        a.d.table[2, 1] = a.bt.pages
    else:
        a.d.shape.max_q = 2
    a.run()
    assert a.d.errors() == -7
    got = a.state()
    for b in (0, 3):
        for x, y in zip(got, right):
            assert torch.equal(x[a.bt.table[b, 0]], y[a.bt.table[b, 0]])


def test_tokens_one_by_one_and_attention_over_them():
    # a sequence appended token by token, then in chunks, and read back: what attention sees is what was stored, and
    # no value is further from its true one than a step of its block's scale
    heads, kvh, dim, page, block = 8, 2, 64, 32, 32
    g = torch.Generator().manual_seed(3)
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda")
    codes = [torch.zeros(4, kvh, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(4, kvh, page // block, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = moe.make_kv_cache_q8(*codes, *scales)
    rope = moe.make_rope(dim, base=1e4)
    held, ks, vs = 0, [], []
    for n in [1] * 20 + [13, 1, 30, 1, 1]:
        held += n
        shape = moe.make_attn_shape(n, 1, heads, kvh, dim, page, 4, 4, n)
        batch = moe.make_attn_batch(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [held])), table)
        ws = torch.zeros(moe.moe_attn_q8_workspace_size(shape, block), dtype=torch.uint8, device="cuda")
        grow = 1.0 + held / 8  # every block's scale grows several times
        q, k, v = (torch.randn(n, h, dim, generator=g).mul(grow).bfloat16().cuda() for h in (heads, kvh, kvh))
        out, lse = torch.empty_like(q), torch.empty(n, heads, device="cuda")
        moe.moe_rope_append_q8(shape, rope, q, k, v, cache, batch, q, workspace=ws)
        moe.moe_paged_attention_q8(shape, q, cache, batch, out, scale=0.05, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert moe.moe_read_device_error(ws) == 0
        f, ms = rates(dim, 1e4)
        ks.append(rotate(k.cpu(), torch.arange(held - n, held), f, ms, False))
        vs.append(v.cpu().double())
    values = [(from_codes(c.cpu()) * power(s.cpu().int() - 127).repeat_interleave(block, 2)[..., None])[table[0].cpu().long()]
              .transpose(0, 1).reshape(kvh, -1, dim)[:, :held] for c, s in zip(codes, scales)]
    steps = [power(s.cpu().int() - 127).repeat_interleave(block, 2)[table[0].cpu().long()].transpose(0, 1).reshape(kvh, -1)[:, :held]
             for s in scales]
    for true, got, s in ((torch.cat(ks), values[0], steps[0]), (torch.cat(vs), values[1], steps[1])):
        true, t = true.transpose(0, 1), got / s[..., None]
        # rounded once when stored and once more each time that the scale grew past it
        assert ((got - true).abs() <= s[..., None] * (step8(t) + 2.0 ** -9 * 4) + 1e-5 * true.abs().amax()).all()
    from attn_ref import Batch
    bt = Batch("bf16", heads, kvh, dim, page, [1], [held], torch.tensor([0, 1]), table.cpu(), 4, q.cpu(),
               *((from_codes(c.cpu()) * power(s.cpu().int() - 127).repeat_interleave(block, 2)[..., None]) for c, s in
                 zip(codes, scales)))
    want, want_lse, tol, tol_lse = attention(bt, 0.05)
    assert ((out.cpu().double() - want).abs() <= tol).all() and ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()
