"""The attention half at its edges on the GPU: refusals that need a device, wrong data that has to be
recorded, values that are not finite, and batches that reach every branch of the schedules."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import FP32, HALF, attention, make_batch, q4_dense  # noqa: E402
from test_gpu_attn import ATTN, NORMAL, SHIFTED, UNIFORM, Dev, check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()


def test_a_call_without_a_workspace_is_refused():
    d = Dev(make_batch(*ATTN["few tokens"], seed=1))
    with pytest.raises(moe.MoEError) as e:
        moe.moe_paged_attention(d.shape, d.q, d.cache, d.batch, d.out)
    assert e.value.status == -4
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rope_append(d.shape, moe.make_rope(128), d.q, d.q[:, :4].contiguous(), d.q[:, 4:].contiguous(), d.cache,
                            d.batch, d.out)
    assert e.value.status == -4


@pytest.mark.parametrize("what", ["negative length", "length past the table", "idle length past the table", "long chunk"])
@pytest.mark.parametrize("tokens", [1, 700])
def test_rope_append_records_what_attention_does(what, tokens):
    # a cache length outside [0, max_pages * page_size], of a sequence without new tokens too, and a chunk
    # past max_q; what the other sequences bring is stored all the same
    q_len, kv_len = [3, 0, tokens, 2], [5, 9, tokens + 1, 4]
    bt = make_batch("bf16", 4, 2, 64, 16, q_len, kv_len, seed=2, fill=5.0)
    d = Dev(bt, max_q=tokens if tokens > 3 else 3)
    x = torch.randn(bt.tokens, 4, 64, device="cuda").bfloat16()
    rope = moe.make_rope(64)
    append = lambda: moe.moe_rope_append(d.shape, rope, x, x[:, :2].contiguous(), x[:, 2:].contiguous(),  # noqa: E731
                                         d.cache, d.batch, d.out, workspace=d.ws)
    append()
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(d.ws) == 0
    first_k = d.k.clone()
    if what == "negative length":
        d.kv_len[2] = -1
    elif what == "length past the table":
        d.kv_len[2] = bt.table.shape[1] * 16 + 1
    elif what == "idle length past the table":
        d.kv_len[1] = bt.table.shape[1] * 16 + 1
    else:
        d.shape.max_q = 2
    d.k.fill_(5.0)
    append()
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(d.ws) == -7
    for b in (0, 3):
        pages = bt.table[b, :-(-kv_len[b] // 16)].long().cuda()
        new = slice(kv_len[b] - q_len[b], kv_len[b])
        rows = lambda c: c[pages].transpose(0, 1).reshape(2, -1, 64)[:, new]  # noqa: E731
        assert torch.equal(rows(d.k), rows(first_k))


@pytest.mark.parametrize("what", ["falls", "first", "idle length", "idle negative length"])
@pytest.mark.parametrize("dtype,dim,most", [("bf16", 128, 1), ("bf16", 64, 40), ("bf16", 128, 40), ("bf16", 96, 3),
                                            ("f32", 64, 40)])
def test_attention_records_wrong_data_of_idle_sequences(what, dtype, dim, most):
    # a cu_q that falls between two sequences or starts late and a wrong length of a sequence without new
    # tokens, by every kernel
    q_len, kv_len = [most, 0, most, 0, 2], [600, 9, most, 3, 700]
    d = Dev(make_batch(dtype, 4, 2, dim, 16, q_len, kv_len, seed=2))
    assert d.attend(0.1) == 0
    if what == "falls":
        d.cu_q[1] = d.cu_q[2] + 1  # the idle one ends before it starts
        d.shape.max_q = d.shape.n_tokens if most > 5 else 2
    elif what == "first":
        d.cu_q[:2] = -3
        d.cu_q[1] = 0
    elif what == "idle length":
        d.kv_len[1] = d.table.shape[1] * 16 + 1
    else:
        d.kv_len[3] = -1
    assert d.attend(0.1) == -7
    assert moe.moe_read_device_error(d.ws) == 0


# batch, one of its sequences and a place among that sequence's new tokens, for each kernel and join
NAN = {"decode in clusters": ("few tokens", 2, 3), "decode in parts": ("decode 400 pairs", 7, 0),
       "decode on the line": ("decode long", 0, 0), "chunks cut": ("chunk over cache", 0, 100),
       "chunks whole": ("chunk ragged", 3, 60), "chunks of heads of 64": ("chunk dim 64", 1, 20),
       "generic alone": ("chunk fp32", 0, 50), "generic in parts": ("head size 256 fp32", 0, 1)}


def _nan_case(name, spoil):
    # `spoil` makes values NaN and returns the rows [tokens][heads] that have to be NaN; the others are right
    spec, b, j = NAN[name]
    bt = make_batch(*ATTN[spec], seed=13)
    out, lse, tol, tol_lse = attention(bt, 0.1)
    nan = spoil(bt, b, j)
    d = Dev(bt)
    assert d.attend(0.1) == 0
    got, got_lse = d.out.cpu().double(), d.lse.cpu().double()
    assert torch.equal(got.isnan().all(-1), nan) and torch.equal(got.isnan().any(-1), nan)
    assert torch.equal(got_lse.isnan(), nan)
    assert ((got - out).abs() <= tol)[~nan].all() and ((got_lse - lse).abs() <= tol_lse)[~nan & lse.isfinite()].all()


@pytest.mark.parametrize("name", list(NAN))
def test_attention_of_a_nan_query_is_nan(name):
    # not 0 with a log-sum of -inf, which says that the token sees no key
    def spoil(bt, b, j):
        t, h = int(bt.cu_q[b]) + j, bt.heads - 1
        bt.q[t, h] = float("nan")
        nan = torch.zeros(bt.tokens, bt.heads, dtype=torch.bool)
        nan[t, h] = True
        return nan
    _nan_case(name, spoil)


@pytest.mark.parametrize("name", [n for n in NAN if n.startswith(("chunks", "generic"))])
def test_attention_of_a_nan_key_is_nan_for_those_who_see_it(name):
    # the key of new token j: the tokens before it do not see it
    def spoil(bt, b, j):
        n, m = bt.q_len[b], bt.kv_len[b]
        p = m - n + j
        bt.k_cache[int(bt.table[b, p // bt.page]), 0, p % bt.page, 3] = float("nan")
        nan = torch.zeros(bt.tokens, bt.heads, dtype=torch.bool)
        t0 = int(bt.cu_q[b])
        nan[t0 + j:t0 + n, :bt.heads // bt.kv_heads] = True
        return nan
    _nan_case(name, spoil)


@pytest.mark.parametrize("dtype,dim,page,tokens", [("bf16", 64, 7, 2), ("bf16", 128, 7, 1), ("bf16", 64, 8, 20),
                                                   ("f32", 8, 7, 1)])
def test_attention_of_nearly_2_to_the_31_keys(dtype, dim, page, tokens):
    # as many keys as a length can say, all on one page but the last, whose scores outweigh the rest: the
    # ends of the ranges of steps and of the masks
    width = (2 ** 31 - 1) // page
    kv, special = width * page, 4  # the last pages hold the new tokens' keys
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(dim)
    k = torch.zeros(special + 1, 1, page, dim)
    k[1:] = 40.0 / dim + 0.02 * torch.randn(special, 1, page, dim, generator=g)
    k, v = k.to(dt), torch.randn(special + 1, 1, page, dim, generator=g).to(dt)
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -special:] = torch.arange(1, special + 1).int()
    q = torch.ones(tokens, 1, dim, dtype=dt, device="cuda")
    shape = moe.make_attn_shape(tokens, 1, 1, 1, dim, page, special + 1, width, tokens, act=dtype)
    batch = moe.make_attn_batch(torch.tensor([0, tokens]).int().cuda(), torch.tensor([kv]).int().cuda(), table)
    ws = torch.zeros(moe.moe_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(tokens, 1, device="cuda")
    moe.moe_paged_attention(shape, q, moe.make_kv_cache(k.cuda(), v.cuda()), batch, out, scale=1.0, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(ws) == 0
    n = special * page
    score = k[1:].double().reshape(n, dim).sum(1)
    hide = torch.arange(n)[None] > torch.arange(n - tokens, n)[:, None]
    total = torch.logsumexp(score.masked_fill(hide, -torch.inf), 1)
    p = torch.exp(score - total[:, None]).masked_fill(hide, 0)
    want = p @ v[1:].double().reshape(n, dim)
    # scores of dim sums of about 40 / dim, twice in a probability; bf16 rounds the probabilities and the result;
    # the keys of score 0 weigh 2^31 e^-40 < 2^-26 together
    err = 2 * (dim + 8) * FP32 * 45 + (HALF["bf16"] if dtype == "bf16" else 0) + (n + 32) * FP32 + 2.0 ** -26
    tol = err * (p @ v[1:].double().abs().reshape(n, dim)) + HALF[dtype] * want.abs() + 2.0 ** -24
    assert ((out.cpu().double()[:, 0] - want).abs() <= tol).all()
    assert ((lse.cpu().double()[:, 0] - total).abs() <= err + 4 * FP32 * total).all()


def _many(seqs, most, keys, long=0):
    """Chunk and cache lengths: up to `most` new tokens and `keys` keys, idle and empty sequences among them, one chunk
    cut short, and one sequence of `long` keys."""
    q = [(i * 7 + i // 5) % (most + 1) for i in range(seqs)]
    kv = [n + (i * 53 + i // 3) % max(keys - n, 1) for i, n in enumerate(q)]
    q[seqs // 3], kv[seqs // 3] = most, most // 2
    q[seqs // 2], kv[seqs // 2] = 1, 0
    if long:
        q[seqs - 2], kv[seqs - 2] = most, long
    return q, kv


# name: dtype, heads, kv_heads, dim, page, (sequences, most new tokens, keys, keys of one)
MANY = {
    "decode even parts 130": ("bf16", 4, 1, 64, 16, (130, 1, 60, 1500)),
    "decode even parts 150": ("bf16", 8, 1, 128, 16, (150, 2, 70, 2500)),
    "decode line 200": ("bf16", 3, 1, 128, 16, (200, 4, 700, 0)),
    "decode line 300": ("bf16", 4, 2, 64, 32, (300, 2, 200, 1200)),
    "decode line 600": ("bf16", 4, 2, 128, 16, (600, 1, 90, 0)),
    "decode one CTA a pair 300": ("bf16", 2, 1, 64, 16, (300, 8, 100, 0)),
    "chunks whole 400": ("bf16", 4, 2, 64, 16, (400, 11, 100, 500)),
    "chunks whole 400 heads of 128": ("bf16", 4, 1, 128, 32, (400, 7, 100, 500)),
    "chunks whole, 17 items a CTA": ("bf16", 4, 2, 64, 16, (1500, 9, 60, 0)),
    "chunks whole, 17 items a CTA, heads of 128": ("bf16", 8, 4, 128, 16, (760, 9, 60, 0)),
    "chunks cut 400": ("bf16", 4, 2, 128, 16, (400, 11, 100, 3000)),
    "chunks cut 500 heads of 64": ("bf16", 6, 2, 64, 16, (500, 9, 300, 2000)),
    "chunks cut, 17 items a CTA": ("bf16", 4, 2, 64, 16, (1600, 9, 40, 700)),
    "chunks cut, 17 items a CTA, heads of 128": ("bf16", 8, 4, 128, 16, (800, 9, 40, 700)),
    "generic 40": ("f32", 3, 1, 24, 16, (40, 9, 90, 0)),
    "generic 150": ("f32", 4, 2, 64, 5, (150, 6, 60, 400)),
    "generic 300": ("bf16", 6, 2, 80, 16, (300, 3, 70, 0)),
}


@pytest.mark.parametrize("name", list(MANY))
def test_attention_of_many_sequences(name):
    # more sequences than one round of a scan takes, and more items a CTA than it lists at a time
    dtype, heads, kv_heads, dim, page, sizes = MANY[name]
    check(make_batch(dtype, heads, kv_heads, dim, page, *_many(*sizes), seed=len(name)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 7, 12, 20, 33])
def test_attention_keeps_its_bits(group, dim):
    # groups that leave rows of a tile empty: what earlier kernels left in shared memory changes nothing
    d = Dev(make_batch("bf16", group, 1, dim, 32, [60, 1, 247], [600, 1, 2315], seed=group, spread=2.0))
    others = [Dev(make_batch("bf16", 8, 1, dim, 32, [300], [900], seed=s, spread=x)) for s, x in enumerate((0.1, 5.0, 50.0))]
    first = None
    for _ in range(4):
        for other in others:
            other.attend(0.3)
            assert d.attend(0.3) == 0
            now = d.out.clone(), d.lse.clone()
            first = now if first is None else first
            assert torch.equal(first[0], now[0]) and torch.equal(first[1], now[1])


@pytest.mark.parametrize("name", ["decode ragged", "chunk over cache", "chunk dim 64", "chunk fp32"])
def test_attention_of_huge_products_and_a_tiny_scale(name):
    # q . k of about 10^35 and a scale of 10^-35: ordinary scores
    bt = make_batch(*ATTN[name], seed=14)
    bt.q *= 2.0 ** 57
    bt.k_cache *= 2.0 ** 57
    check(bt, scale=2.0 ** -117)


# ------------------------------------------------------------------------------- 4-bit linear

# nearly uniform: two small values off by 2^-18 of themselves; computed in fp32 steps; a zero that rounding missed
BENT = [v * (1 + 2.0 ** -18) if j in (7, 8) else v for j, v in enumerate(UNIFORM)]
BOOKS = {"bent": BENT, "steps": torch.linspace(-1, 1, 16).tolist(), "zero": [0.125 * (j - 5) + (j == 5) * 1e-16 for j in range(16)]}


@pytest.mark.parametrize("book", list(BOOKS))
@pytest.mark.parametrize("T,K,N,q_block", [(7, 512, 300, 64), (16, 192, 2000, 32), (12, 640, 20000, 64), (20, 2048, 4200, 64)])
def test_q4_linear_keeps_nearly_uniform_values(T, K, N, q_block, book):
    # rows of x with a single one: each fp32 result is one weight.  A codebook value is held to 2^-20, its product
    # with the scale and the sum of its parts round a few times more
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    scales = (torch.rand(N, K // q_block, generator=g) + 0.25).bfloat16()
    x = torch.zeros(T, K)
    x[torch.arange(T), torch.randperm(K, generator=g)[:T]] = 1.0
    values = [float(torch.tensor(v).float()) for v in BOOKS[book]]
    want = x.double() @ q4_dense(codes, scales, values, q_block).T
    shape, weight = moe.make_q4_linear_shape(T, K, N, "f32", q_block), moe.make_q4_weight(codes.cuda(), scales.cuda(), values)
    out = torch.empty(T, N, device="cuda")
    moe.moe_q4_linear(shape, x.bfloat16().cuda(), weight, out)
    over = (out.cpu().double() - want).abs() - (2.0 ** -20 + 6 * FP32) * want.abs()
    assert (over <= 1e-12).all(), over.max()


@pytest.mark.parametrize("book", [UNIFORM, NORMAL, SHIFTED], ids=["uniform", "normal", "shifted"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,q_block", [(1, 2048, 640, 64), (7, 512, 300, 32), (12, 640, 20000, 64), (8, 8192, 64, 64),
                                           (20, 2048, 4200, 64), (40, 4096, 2112, 128), (5, 240, 31, 48)])
def test_q4_linear_of_infinite_and_huge_inputs(T, K, N, q_block, out, book):
    # by the definition: an infinite x gives infinities (NaN where the weight is 0, or two cancel), one past 2^123 a
    # finite sum, NaN NaN; the other rows are what they are
    g = torch.Generator().manual_seed(K + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    scales = (torch.rand(N, K // q_block, generator=g) * 0.1 + 0.05).bfloat16()
    x = torch.randn(T, K, generator=g).bfloat16()
    inf = float("inf")
    for t, special in enumerate([[inf], [-inf, inf], [2.0 ** 126], [float("nan")], [-(2.0 ** 124), 2.0 ** 125]]):
        if t < T:
            for i, v in enumerate(special):
                x[t, (37 * t + 61 * i + K // 2) % K] = v
    values = [float(torch.tensor(v).float()) for v in book]
    w = q4_dense(codes, scales, values, q_block)
    want, size = x.double() @ w.T, x.double().abs() @ w.abs().T
    shape, weight = moe.make_q4_linear_shape(T, K, N, out, q_block), moe.make_q4_weight(codes.cuda(), scales.cuda(), values)
    buf = torch.empty(T, N, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    moe.moe_q4_linear(shape, x.cuda(), weight, buf)
    got = buf.cpu().double()
    assert torch.equal(got.isnan(), want.isnan())
    at_inf = want.isinf()
    assert torch.equal(got[at_inf], want[at_inf]) and not got[~at_inf].isinf().any()
    # as for finite inputs: K products and sums in fp32, a codebook value held to 2^-17, one rounding
    tol = size * (K + 16) * FP32 + size * 2.0 ** -17 + (HALF[out] + FP32) * want.abs()
    at = want.isfinite()
    assert ((got - want).abs() <= tol)[at].all()
