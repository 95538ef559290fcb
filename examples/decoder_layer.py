"""One decoder layer with 4-bit weights, served from a paged cache: the attention half
(moe_q4_linear, moe_rope_append, moe_paged_attention) around the MoE block
(moe_forward_rmsnorm), for prompts in chunks and for single tokens.  The cache holds 16-bit values or
8-bit ones (moe_rope_append_q8, moe_paged_attention_q8), and the layer sees all keys or a window and a few first ones
(moe_paged_attention_window).

    python examples/decoder_layer.py

builds layers with random weights, runs two requests' prompts in chunks of different
lengths, then a few decode steps captured in a CUDA graph, and prints what a step takes: with a 16-bit cache, then
with an 8-bit one and a window.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_routing_grouped_router_gb300 as moe  # noqa: E402
from top_routing_grouped_router_gb300 import build  # noqa: E402

CODEBOOK = [-1 + 2 * j / 15 for j in range(16)]
GROUP = 64


def random_q4(g, *shape):
    """Random codes and scales of a [..., rows, cols] matrix whose products keep their inputs' size."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8)
    level = math.sqrt(sum(c * c for c in CODEBOOK) / 16 * shape[-1])
    scales = (0.5 + torch.rand(*shape[:-1], shape[-1] // GROUP, generator=g, device="cuda")) / level
    return codes, scales.bfloat16()


class DecoderLayer:
    """Weights, cache and workspaces of one layer; `step` runs it on new tokens of any of its sequences."""

    def __init__(self, hidden=2048, heads=32, kv_heads=4, dim=128, experts=128, top_k=8, inner=768, pages=256,
                 page_size=16, max_seqs=8, max_pages=64, rope_base=1e6, seed=0, scale_block=None, window=None, sinks=0):
        """scale_block: None for a 16-bit cache, or the tokens that share a scale of an 8-bit one; window: None, or how many
        keys a token sees up to its own, beside the sequence's first `sinks`."""
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.experts, self.top_k, self.inner, self.eps = experts, top_k, inner, 1e-6
        self.page_size, self.pages, self.max_pages = page_size, pages, max_pages
        ones = lambda n: (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16()  # noqa: E731
        self.norm1, self.norm2 = ones(hidden), ones(hidden)
        self.qkv_cols = (heads + 2 * kv_heads) * dim
        self.w_qkv = moe.make_q4_weight(*random_q4(g, self.qkv_cols, hidden), CODEBOOK)
        self.w_out = moe.make_q4_weight(*random_q4(g, hidden, heads * dim), CODEBOOK)
        self.rope = moe.make_rope(dim, base=rope_base, q_gamma=ones(dim), k_gamma=ones(dim), eps=self.eps)
        self.w_router = (torch.randn(experts, hidden, generator=g, device="cuda") / math.sqrt(hidden)).bfloat16()
        gate, up, down = (random_q4(g, experts, r, c) for r, c in ((inner, hidden), (inner, hidden), (hidden, inner)))
        self.gate, self.up, self.down = gate[0], up[0], down[0]
        self.expert_scales = gate[1], up[1], down[1]
        self.q4 = moe.MoEQ4(*(s.data_ptr() for s in self.expert_scales), (moe.MoEQ4._fields_[3][1])(*CODEBOOK))
        self.scale_block, self.window = scale_block, moe.make_attn_window(window, sinks) if window else None
        zeros = lambda dtype, *s: [torch.zeros(pages, kv_heads, *s, dtype=dtype, device="cuda") for _ in range(2)]  # noqa: E731
        if scale_block:
            self.cache = moe.make_kv_cache_q8(*zeros(torch.float8_e4m3fn, page_size, dim), *zeros(torch.uint8, page_size // scale_block))
        else:
            self.cache = moe.make_kv_cache(*zeros(torch.bfloat16, page_size, dim))
        # the host's view of the cache: which pages a sequence holds, and how many keys
        self.free = list(range(pages))
        self.lengths = [0] * max_seqs
        self.table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32)

    def reserve(self, seq, tokens):
        """Pages for `tokens` more keys of a sequence."""
        held, need = -(-self.lengths[seq] // self.page_size), -(-(self.lengths[seq] + tokens) // self.page_size)
        if need > self.max_pages or need - held > len(self.free):
            raise RuntimeError("the cache is full")
        for i in range(held, need):
            self.table[seq, i] = self.free.pop()
        self.lengths[seq] += tokens

    def plan(self, chunks):
        """What a step on chunks {sequence: new tokens} needs beside its input rows (which hold the sequences' tokens
        one after another): reserves the cache, makes the batch, the shapes, the workspaces and the buffers."""
        seqs, counts = list(chunks), list(chunks.values())
        for s, n in chunks.items():
            self.reserve(s, n)
        n = sum(counts)
        p = {"tokens": n}
        p["batch"] = moe.make_attn_batch(torch.tensor([0] + counts).cumsum(0).int().cuda(),
                                         torch.tensor([self.lengths[s] for s in seqs], dtype=torch.int32, device="cuda"),
                                         self.table[seqs].cuda())
        p["attn"] = moe.make_attn_shape(n, len(seqs), self.heads, self.kv_heads, self.dim, self.page_size, self.pages,
                                        self.max_pages, max(counts))
        p["moe"] = moe.make_shape(n, self.hidden, self.experts, self.top_k, self.inner, "bf16", "q4", q_block=GROUP)
        p["in"] = moe.make_q4_linear_shape(n, self.hidden, self.qkv_cols, q_block=GROUP)
        p["out"] = moe.make_q4_linear_shape(n, self.heads * self.dim, self.hidden, q_block=GROUP)
        size = moe.moe_attn_q8_workspace_size(p["attn"], self.scale_block) if self.scale_block else moe.moe_attn_workspace_size(p["attn"])
        p["attn_ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        p["moe_ws"] = torch.zeros(moe.moe_workspace_size(p["moe"]), dtype=torch.uint8, device="cuda")
        buf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        p["qkv"], p["o"] = buf(n, self.qkv_cols), buf(n, self.heads, self.dim)
        p["hs"], p["y"] = buf(n, self.hidden), buf(n, self.hidden)
        return p

    def step(self, p, x):
        """The layer on the plan's new tokens, x [tokens][hidden] bf16; returns the plan's output rows."""
        n, hq, hk, d = p["tokens"], self.heads, self.kv_heads, self.dim
        xn = (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + self.eps) * self.norm1.float()).bfloat16()
        moe.moe_q4_linear(p["in"], xn, self.w_qkv, p["qkv"])
        q, k, v = p["qkv"].split([hq * d, hk * d, hk * d], 1)
        q, k, v = q.view(n, hq, d), k.view(n, hk, d), v.view(n, hk, d)
        append = moe.moe_rope_append_q8 if self.scale_block else moe.moe_rope_append
        append(p["attn"], self.rope, q, k, v, self.cache, p["batch"], q, workspace=p["attn_ws"])
        if self.scale_block:
            moe.moe_paged_attention_q8(p["attn"], q, self.cache, p["batch"], p["o"], window=self.window, workspace=p["attn_ws"])
        elif self.window:
            moe.moe_paged_attention_window(p["attn"], q, self.cache, p["batch"], self.window, p["o"], workspace=p["attn_ws"])
        else:
            moe.moe_paged_attention(p["attn"], q, self.cache, p["batch"], p["o"], workspace=p["attn_ws"])
        moe.moe_q4_linear(p["out"], p["o"].view(n, hq * d), self.w_out, p["hs"], residual=x)
        moe.moe_forward_rmsnorm(p["moe"], p["hs"], self.norm2, self.eps, self.w_router, None, self.gate, self.up, self.down,
                                self.q4, p["y"], workspace=p["moe_ws"])
        return p["y"]

    def errors(self, p):
        """Device-side error codes of the attention half (its projections, then the plan's workspace) and of the MoE
        half (0: none); synchronises.  The projections' word is one for all streams of the device."""
        linear, attn = moe.moe_q4_linear_read_error(), moe.moe_read_device_error(p["attn_ws"])
        return linear or attn, moe.moe_read_device_error(p["moe_ws"])


def serve(what, **kw):
    layer = DecoderLayer(**kw)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = lambda n: torch.randn(n, layer.hidden, generator=g, device="cuda").bfloat16()  # noqa: E731
    for chunks in ({0: 100, 1: 37}, {0: 60}):  # the prompts, the longer one in two chunks
        p = layer.plan(chunks)
        layer.step(p, rows(p["tokens"]))
        print(what, "chunks", chunks, "errors", layer.errors(p))
    p, x = layer.plan({0: 1, 1: 1}), rows(2)  # a decode step
    layer.step(p, x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.step(p, x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print("%s: decode step of 2 sequences %.1f us, errors %s" % (what, start.elapsed_time(end) * 10, layer.errors(p)))


def main():
    build.build()
    serve("16-bit cache")
    serve("8-bit cache, window of 64", scale_block=16, window=64, sinks=4)


if __name__ == "__main__":
    main()
