"""The 8-bit cache and attention with a window in 64 bits on the CPU, from their definitions, and the error
bounds of the kernels' arithmetic (used by the GPU tests)."""
from __future__ import annotations

import math

import torch

from attn_ref import FP32, HALF, Batch, keys_of

LARGEST, LOWEST, HIGHEST = 448.0, -110, 119


def exponents(top):
    """The smallest e with top <= 448 2^e, within what an append writes."""
    m, e = torch.frexp(top.double())  # top = m 2^e, m in [1/2, 1); 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, e, torch.full_like(e, LOWEST)).clamp(LOWEST, HIGHEST)


def power(e):
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)


def step8(x):
    """The distance of neighbouring e4m3 values around x."""
    _, e = torch.frexp(x.double())
    return power((e - 4).clamp(min=-9))


def round8(x):
    """The nearest e4m3 values, ties to even, |x| <= 448; 64 bits."""
    return torch.round(x / step8(x)) * step8(x)


def to_codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def from_codes(codes):
    return codes.view(torch.float8_e4m3fn).double()


def store(cache, block):
    """A cache [pages][heads][slots][dim] in 8 bits: (codes, bytes, the values that they stand for in 64 bits).  What is
    not finite becomes NaN."""
    pages, heads, slots, dim = cache.shape
    x = cache.double().view(pages, heads, slots // block, block, dim)
    x = torch.where(x.isfinite(), x, torch.full_like(x, math.nan))
    e = exponents(x.abs().nan_to_num(nan=0.0).amax((3, 4)))
    s = power(e)[..., None, None]
    codes = to_codes((x / s).float()).view(pages, heads, slots // block, block, dim)
    return codes.view(cache.shape), (e + 127).to(torch.uint8), (from_codes(codes) * s).view(cache.shape)


def attention(bt: Batch, scale, window=None, sinks=0):
    """(out, lse, bound on |out - kernel's out|, bound on |lse - kernel's|) of a batch whose tokens see a window (None:
    all keys) and the first keys; 64 bits.  The bounds are attn_ref's, over the keys that a row sees."""
    out = torch.zeros(bt.tokens, bt.heads, bt.dim, dtype=torch.float64)
    lse = torch.full((bt.tokens, bt.heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    group = bt.heads // bt.kv_heads
    for b, (n, m) in enumerate(zip(bt.q_len, bt.kv_len)):
        if n == 0 or m == 0:
            continue
        t0 = int(bt.cu_q[b])
        place, key = torch.arange(m - n, m)[:, None], torch.arange(m)[None]
        seen = key <= place
        if window is not None:
            seen &= (place - key < window) | (key < sinks)
        k, v = keys_of(bt, b, bt.k_cache), keys_of(bt, b, bt.v_cache)
        used = seen.any(0)
        k, v = (torch.where(used[None, :, None], x, torch.zeros(())) for x in (k, v))
        q = bt.q[t0:t0 + n].double().view(n, bt.kv_heads, group, bt.dim).permute(1, 2, 0, 3)
        s = (q @ k.transpose(1, 2)[:, None] * scale).masked_fill(~seen, -math.inf)
        total = torch.logsumexp(s, 3)
        p = torch.nan_to_num(torch.exp(s - total[..., None]), nan=0.0)
        o, size_v = p @ v[:, None], p @ v.abs()[:, None]
        size = (q.abs() @ k.abs().transpose(1, 2)[:, None] * abs(scale)).masked_fill(~seen, 0).amax(3)
        ds = (bt.dim + 8) * FP32 * size
        dp = 2 * ds + (m + 32) * FP32 + (HALF["bf16"] if bt.dtype == "bf16" else 0)
        back = lambda x: x.permute(2, 0, 1, *range(3, x.dim())).reshape(n, bt.heads, *x.shape[3:])  # noqa: E731
        rows = slice(t0, t0 + n)
        out[rows], lse[rows] = back(o), back(total)
        tol[rows] = back(dp[..., None] * size_v + HALF[bt.dtype] * o.abs() + 1e-30)
        tol_lse[rows] = back(torch.where(total.isinf(), torch.zeros(()), ds + (m + 32) * FP32 + 4 * FP32 * total.abs()))
    return out, lse, tol, tol_lse
