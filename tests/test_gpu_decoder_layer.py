"""The example's decoder layer: prompts in one chunk, in several, and token by token give the
same rows, and its attention half agrees with 64 bits."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

SIZES = dict(hidden=256, heads=8, kv_heads=2, dim=64, experts=8, top_k=2, inner=128, pages=40, page_size=16, max_seqs=3,
             max_pages=12)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()
    import decoder_layer
    return decoder_layer


def _attention_half(layer, x):
    """hs = x + attention(x) of one sequence from its start, 64 bits, from the weights' values."""
    from attn_ref import q4_dense, rates, rotate
    x = x.cpu().double()
    n, hq, hk, d = x.shape[0], layer.heads, layer.kv_heads, layer.dim
    w = [q4_dense(t.tensors[0].cpu(), t.tensors[1].cpu(), [float(torch.tensor(c).float()) for c in
         (-1 + 2 * j / 15 for j in range(16))], 64) for t in (layer.w_qkv, layer.w_out)]
    xn = x / torch.sqrt(x.square().mean(1, keepdim=True) + layer.eps) * layer.norm1.cpu().double()
    q, k, v = (xn @ w[0].T).split([hq * d, hk * d, hk * d], 1)
    f, ms = rates(d, 1e6)
    pos = torch.arange(n)
    q = rotate(q.view(n, hq, d), pos, f, ms, False, layer.rope.tensors[1].cpu())
    k = rotate(k.view(n, hk, d), pos, f, ms, False, layer.rope.tensors[2].cpu()).repeat_interleave(hq // hk, 1)
    v = v.view(n, hk, d).repeat_interleave(hq // hk, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) / d ** 0.5
    p = s.masked_fill(torch.ones(n, n).triu(1).bool(), -torch.inf).softmax(-1)
    o = torch.einsum("hqk,khd->qhd", p, v).reshape(n, hq * d)
    return x + o @ w[1].T


@pytest.mark.parametrize("pieces", [[50], [20, 30], [33, 16, 1], [1] * 12])
def test_chunks_agree_with_64_bits(example, pieces):
    layer = example.DecoderLayer(**SIZES, seed=4)
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
    want = _attention_half(layer, x)
    # five roundings to bf16 on the way (normed rows, qkv, rotated q and k, probabilities, output) and
    # that of the sum, each half a step (2^-8) of values of the rows' size, through softmax (twice)
    err = (torch.cat(got).cpu().double() - want).norm() / want.norm()
    assert err <= 8 * 2.0 ** -8, err


def test_decode_graph_and_moe_output(example):
    # a captured decode step equals the eager one bit for bit, the MoE half included
    layer = example.DecoderLayer(**SIZES, seed=5)
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


def test_a_full_cache_is_refused(example):
    layer = example.DecoderLayer(**SIZES)
    with pytest.raises(RuntimeError):
        layer.plan({0: SIZES["page_size"] * SIZES["max_pages"] + 1})


def test_a_failed_projection_is_an_error(example):
    # a projection whose tensor-core kernel gave up (its operands can never be complete) shows in errors()
    import top_routing_grouped_router_gb300 as moe
    layer = example.DecoderLayer()
    p = layer.plan({0: 20})
    x = torch.zeros(20, layer.hidden, dtype=torch.bfloat16, device="cuda")
    moe.moe_debug_set_waits(1_000_000, 1)
    try:
        moe.moe_q4_linear(p["in"], x, layer.w_qkv, p["qkv"])
        torch.cuda.synchronize()
    finally:
        moe.moe_debug_set_waits()
    assert layer.errors(p) == (-7, 0)
    layer.step(p, x)
    assert layer.errors(p) == (0, 0)
