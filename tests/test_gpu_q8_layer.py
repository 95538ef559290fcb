"""The 8-bit cache and the window as they are used: a whole layer's steps, in stream order, captured, and after a
wait that ran out."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import make_batch  # noqa: E402
from q8_ref import attention  # noqa: E402
from test_gpu_attn_order import Writer  # noqa: E402
from test_gpu_decoder_layer import SIZES  # noqa: E402
from test_gpu_q8_cache import APPEND, BATCH, Append, Dev  # noqa: E402


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()
    import decoder_layer
    return decoder_layer


def _attention_half(layer, x, window, sinks):
    """hs = x + attention(x) of one sequence from its start, 64 bits, from the weights' values, with unrounded k and v."""
    from attn_ref import q4_dense, rates, rotate
    x = x.cpu().double()
    n, hq, hk, d = x.shape[0], layer.heads, layer.kv_heads, layer.dim
    w = [q4_dense(t.tensors[0].cpu(), t.tensors[1].cpu(), [float(torch.tensor(c).float()) for c in
         (-1 + 2 * j / 15 for j in range(16))], 64) for t in (layer.w_qkv, layer.w_out)]
    xn = x / torch.sqrt(x.square().mean(1, keepdim=True) + layer.eps) * layer.norm1.cpu().double()
    q, k, v = (xn @ w[0].T).split([hq * d, hk * d, hk * d], 1)
    f, _ = rates(d, 1e6)
    pos = torch.arange(n)
    q = rotate(q.view(n, hq, d), pos, f, 1.0, False, layer.rope.tensors[1].cpu())
    k = rotate(k.view(n, hk, d), pos, f, 1.0, False, layer.rope.tensors[2].cpu()).repeat_interleave(hq // hk, 1)
    v = v.view(n, hk, d).repeat_interleave(hq // hk, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) / d ** 0.5
    seen = (pos[None] <= pos[:, None]) & ((pos[:, None] - pos[None] < (window or n)) | (pos[None] < sinks))
    o = torch.einsum("hqk,khd->qhd", s.masked_fill(~seen, -torch.inf).softmax(-1), v).reshape(n, hq * d)
    return x + o @ w[1].T


@pytest.mark.parametrize("block,window,sinks", [(16, None, 0), (8, 11, 2), (None, 11, 2), (None, 1, 0), (16, 40, 0)])
@pytest.mark.parametrize("pieces", [[50], [20, 30], [33, 16, 1], [1] * 12])
def test_layer_agrees_with_64_bits(example, pieces, block, window, sinks):
    layer = example.DecoderLayer(**SIZES, seed=4, scale_block=block, window=window, sinks=sinks)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    n = sum(pieces)
    x, other = (torch.randn(n, layer.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    got, at = [], 0
    for c in pieces:  # the sequence and another one in every step
        p = layer.plan({2: c, 0: c})
        layer.step(p, torch.cat([x[at:at + c], other[at:at + c]]))
        assert layer.errors(p) == (0, 0)
        got.append(p["hs"][:c].clone())
        at += c
    want = _attention_half(layer, x, window, sinks)
    # five roundings to bf16 on the way (normed rows, qkv, rotated q and k, probabilities, output) and that of the sum,
    # each half a step (2^-8) of values of the rows' size, through softmax (twice); k and v in 8 bits are off by 2^-4 at
    # most each (rounded again where a block's scale grows: twice that), k through softmax twice
    err = (torch.cat(got).cpu().double() - want).norm() / want.norm()
    assert err <= 8 * 2.0 ** -8 + (6 * 2.0 ** -4 if block else 0), err


@pytest.mark.parametrize("block,window", [(16, None), (16, 9), (None, 9)])
def test_decode_graph(example, block, window):
    # a captured decode step equals the eager one bit for bit
    layer = example.DecoderLayer(**SIZES, seed=5, scale_block=block, window=window, sinks=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    rows = lambda n: torch.randn(n, layer.hidden, generator=g, device="cuda").bfloat16()  # noqa: E731
    p = layer.plan({0: 30, 1: 9})
    layer.step(p, rows(39))
    p, x = layer.plan({0: 1, 1: 1}), rows(2)
    eager = layer.step(p, x).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(p, x)
    p["y"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p["y"], eager) and torch.isfinite(eager).all()
    assert layer.errors(p) == (0, 0)


KERNELS = {"decode": "decode ragged", "decode many rows": "decode group 16", "chunk": "chunk over cache", "chunk dim 64": "chunk dim 64",
           "generic": "chunk fp32"}


@pytest.mark.parametrize("name", list(KERNELS))
@pytest.mark.parametrize("block", [None, 16])
def test_attention_reads_what_the_kernel_before_wrote(example, name, block):
    bt = make_batch(*BATCH[KERNELS[name]], seed=3)
    d = Dev(bt, block)
    target = d.q[bt.tokens - 1, 0, :8]
    old, write = target.clone(), Writer(target)
    d.attend(0.1, 300, 2)
    torch.cuda.synchronize()
    stale = d.out.clone()
    write()
    torch.cuda.synchronize()
    d.attend(0.1, 300, 2)
    assert d.errors() == 0
    want = d.out.clone()
    assert not torch.equal(want, stale)
    for _ in range(3):
        target.copy_(old)
        torch.cuda.synchronize()
        write()
        d.attend(0.1, 300, 2)
        assert d.errors() == 0 and torch.equal(d.out, want)


@pytest.mark.parametrize("name", ["decode", "prompt", "interleaved part"])
@pytest.mark.parametrize("what", ["k", "v", "q"])
def test_append_reads_what_the_kernel_before_wrote(example, name, what):
    a = Append(APPEND[name], seed=2)
    target = getattr(a, what)[a.bt.tokens - 1, 0, :8]
    old, write = target.clone(), Writer(target)
    result = lambda: [a.d.out.clone().cpu(), *a.state()]  # noqa: E731
    before = a.state()
    a.run()
    torch.cuda.synchronize()
    stale = result()

    def back():
        target.copy_(old)
        for x, y in zip((a.d.k, a.d.ks, a.d.v, a.d.vs), before):
            x.copy_(y)
        torch.cuda.synchronize()

    back()
    write()
    torch.cuda.synchronize()
    a.run()
    assert a.d.errors() == 0
    want = result()
    assert not all(torch.equal(x, y) for x, y in zip(want, stale))
    for _ in range(3):
        back()
        write()
        a.run()
        assert a.d.errors() == 0 and all(torch.equal(x, y) for x, y in zip(result(), want))


@pytest.mark.parametrize("name", ["chunk over cache", "chunk dim 64", "chunk ragged"])
@pytest.mark.parametrize("block", [None, 16])
def test_a_wait_that_runs_out(example, name, block):
    # the softmax's arrivals can never be enough: the waits end after their limit with an error recorded, and the next
    # ordinary call is right
    bt = make_batch(*BATCH[name], seed=7)
    d = Dev(bt, block)
    moe.moe_debug_set_waits(1_000_000, 1)
    try:
        d.attend(0.1, 10**6, 1)
        assert d.errors() == -7
    finally:
        moe.moe_debug_set_waits()
    for window in (None if block else 10**6, 100):
        d.attend(0.1, window, 1)
        assert d.errors() == 0
        out, _, tol, _ = attention(bt, 0.1, window, 1)
        assert ((d.out.cpu().double() - out).abs() <= tol).all()


@pytest.mark.parametrize("block", [None, 16])
@pytest.mark.parametrize("dtype,dim,page,tokens", [("bf16", 64, 16, 2), ("bf16", 128, 16, 20), ("f32", 16, 16, 1)])
def test_windows_at_the_end_of_nearly_2_to_the_31_keys(example, block, dtype, dim, page, tokens):
    # as many keys as a length can say, nearly all on one page: the ends of the ranges of steps, masks and places
    width = (2 ** 31 - 1) // page
    kv, special, sinks = width * page, 8, 5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(dim)
    k, v = (torch.randn(special + 1, 1, page, dim, generator=g).to(dt) for _ in range(2))
    table = torch.full((1, width), 1 << 30, dtype=torch.int32, device="cuda")  # what no token sees is not read
    table[0, 0] = 0
    table[0, -special:] = torch.arange(1, special + 1).int()
    q = torch.randn(tokens, 2, dim, generator=g).to(dt).cuda()
    shape = moe.make_attn_shape(tokens, 1, 2, 1, dim, page, special + 1, width, tokens, act=dtype)
    batch = moe.make_attn_batch(torch.tensor([0, tokens]).int().cuda(), torch.tensor([kv]).int().cuda(), table)
    window = special * page - tokens  # of the first token: within the special pages
    out, lse = torch.empty_like(q), torch.empty(tokens, 2, device="cuda")
    w = moe.make_attn_window(window, sinks)
    if block:
        from q8_ref import store
        (kc, ks, k), (vc, vs, v) = store(k, block), store(v, block)
        ws = torch.zeros(moe.moe_attn_q8_workspace_size(shape, block), dtype=torch.uint8, device="cuda")
        moe.moe_paged_attention_q8(shape, q, moe.make_kv_cache_q8(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()), batch, out, window=w,
                                   scale=0.3, lse=lse, workspace=ws)
    else:
        ws = torch.zeros(moe.moe_attn_workspace_size(shape), dtype=torch.uint8, device="cuda")
        moe.moe_paged_attention_window(shape, q, moe.make_kv_cache(k.cuda(), v.cuda()), batch, w, out, scale=0.3, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert moe.moe_read_device_error(ws) == 0
    # the same batch without the keys between
    from attn_ref import Batch
    n = page + special * page
    bt = Batch(dtype, 2, 1, dim, page, [tokens], [n], torch.tensor([0, tokens]), torch.arange(special + 1).int()[None], special + 1,
               q.cpu(), k, v)
    want, want_lse, tol, tol_lse = attention(bt, 0.3, window, sinks)
    assert ((out.cpu().double() - want).abs() <= tol).all() and ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()
