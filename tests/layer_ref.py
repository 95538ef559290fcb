"""The attention half of examples/decoder_layer.py in 64 bits, in two parts that are compared apart: what a step writes into
the cache, and what attention adds to the residual over the cache as it lies there (used by the CPU and GPU tests)."""
from __future__ import annotations

import dataclasses

import torch

from attn_ref import q4_dense, rates, rotate

BF16, F16 = torch.bfloat16, torch.float16
BASE = 1e6


@dataclasses.dataclass
class Half:
    heads: int
    kv_heads: int
    dim: int
    norm: torch.Tensor
    q_norm: torch.Tensor
    k_norm: torch.Tensor
    w_qkv: torch.Tensor
    w_out: torch.Tensor
    eps: float = 1e-6

    @classmethod
    def of(cls, layer):
        book = [float(torch.tensor(-1 + 2 * j / 15).float()) for j in range(16)]
        w = [q4_dense(t.tensors[0].cpu(), t.tensors[1].cpu(), book, 64) for t in (layer.w_qkv, layer.w_out)]
        return cls(layer.heads, layer.kv_heads, layer.dim, layer.norm1.cpu().double(), layer.rope.tensors[1].cpu(),
                   layer.rope.tensors[2].cpu(), *w, layer.eps)


def _rounded(x, on, dtype=BF16):
    return x.to(dtype).double() if on else x


def heads_of(h: Half, x, first, rounded, turn=True):
    """q, k, v of the tokens x [n][hidden] from place `first` on; rounded: to bf16 where the layer does that (normed rows,
    the projection's output, q)."""
    x = x.double()
    n = len(x)
    xn = _rounded(x / torch.sqrt(x.square().mean(1, keepdim=True) + h.eps) * h.norm, rounded)
    qkv = _rounded(xn @ h.w_qkv.T, rounded)
    q, k, v = qkv.split([h.heads * h.dim, h.kv_heads * h.dim, h.kv_heads * h.dim], 1)
    f, _ = rates(h.dim, BASE)
    places = torch.arange(first, first + n) if turn else torch.zeros(n)
    q = _rounded(rotate(q.reshape(n, -1, h.dim), places, f, 1.0, False, h.q_norm), rounded)
    return q, rotate(k.reshape(n, -1, h.dim), places, f, 1.0, False, h.k_norm), v.reshape(n, -1, h.dim)


def added(h: Half, x, q, k, v, first, window, sinks, rounded, scale=1.0, later=0):
    """attention's part of hs - x for the tokens x at places first .. over the sequence's k, v [keys][kv heads][dim];
    rounded: probabilities to this type, o and hs to bf16.  scale, later: planted mistakes of the softmax's factor, the mask."""
    n, m, group = len(q), len(k), h.heads // h.kv_heads
    place, key = torch.arange(first, first + n)[:, None], torch.arange(m)[None]
    seen = key <= place + later
    if window is not None:
        seen &= (place - key < window) | (key < sinks)
    s = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(group, 1)) * (scale / h.dim ** 0.5)
    s = s.masked_fill(~seen, -torch.inf)
    p = torch.exp(s - s.amax(2, keepdim=True))
    r = _rounded(p, rounded is not None, rounded)
    o = torch.einsum("hqk,khd->qhd", r / p.sum(2, keepdim=True), v.repeat_interleave(group, 1)).reshape(n, -1)
    a = _rounded(o, rounded is not None) @ h.w_out.T
    return a if rounded is None else _rounded(x.double() + a, True) - x.double()


def bound(h: Half, x, k, v, first, window, sinks, eight_bit):
    """(what attention adds, by the definition; how far a layer that rounds where this one does may be from it, as the norm of the
    difference).  The roundings are made in 64 bits at the layer's places, which gives an error of the same size as the kernels':
    independent ones over a few thousand elements, whose norm scatters by a few per cent.  Twice that leaves room for
    fp32's sums and for values that round to the other side."""
    want = added(h, x, heads_of(h, x, first, False)[0], k, v, first, window, sinks, None)
    near = added(h, x, heads_of(h, x, first, True)[0], k, v, first, window, sinks, F16 if eight_bit else BF16)
    return want, 2 * (near - want).norm()


def cache_bound(eight_bit):
    """How far the cache's values may be from k and v, relative to these, as a norm: half a step of e4m3 (2^-4 of a value; a
    value whose block's scale grows stays what it is unless it is small) or of bf16, and the roundings of the normed rows and of
    the projection's output."""
    return (2.0 ** -4 if eight_bit else 2.0 ** -8) + 3 * 2.0 ** -8
