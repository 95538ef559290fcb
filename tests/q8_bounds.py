"""Bounds of attention over the 8-bit cache from what its kernels round: probabilities to fp16, not to bf16 as over a 16-bit
cache (used by the CPU and GPU tests)."""
from __future__ import annotations

import math

import torch

from attn_ref import FP32, HALF, Batch, keys_of

F16 = 2.0 ** -11  # half a step of fp16 relative to the value


def attention8(bt: Batch, scale, window=None, sinks=0, probabilities=None):
    """(out, bound on |out - kernel's out|) in 64 bits.  `probabilities`: a type that the largest-based probabilities
    2^(s - max) are rounded to on the way, as a kernel would (for the tests of the bound itself).

    A probability is off by two scores' errors and its part in a sum of m terms, as in attn_ref, and by half a step of fp16.
    Small ones are off by half of fp16's smallest step instead, 2^-25, of what the kernels make of them.  Chunks: times 2^7 (2^-32
    of its value for each key), and what a block's scale is less than 2^-15 of 2^-7 of the largest at hand (2^-54 of the largest
    value that a block can hold, 448 of its scale).  Decode, up to 16 query rows a key head: times 2^14 and the difference of its
    block's scale to the largest at hand (2^-39 of the largest value; or, as the unit follows a step's scale within 2^6, 2^-33 of its own).  A k far below the largest of 128 keys loses what lies under 2^-40 of that."""
    out = torch.zeros(bt.tokens, bt.heads, bt.dim, dtype=torch.float64)
    tol = torch.zeros_like(out)
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
        top = s.amax(3, keepdim=True)
        e = torch.nan_to_num(torch.exp(s - top), nan=0.0)
        total = e.sum(3, keepdim=True).clamp(min=1e-300)
        r = e if probabilities is None else e.to(probabilities).double()
        o, size_v = r / total @ v[:, None], e / total @ v.abs()[:, None]
        size = (q.abs() @ k.abs().transpose(1, 2)[:, None] * abs(scale)).masked_fill(~seen, 0).amax(3)
        ds = (bt.dim + 8) * FP32 * size
        if bt.dtype == "bf16":
            ds = ds + abs(scale) * q.abs().sum(3) * k.abs().amax((1, 2))[:, None, None] * 2 * 2.0 ** -40
        dp = 2 * ds + (m + 32) * FP32 + (F16 if bt.dtype == "bf16" else 0)
        t = dp[..., None] * size_v + HALF[bt.dtype] * o.abs() + 1e-30
        if bt.dtype == "bf16":
            count = seen.double()
            largest = 2 * v.abs().amax((1, 2))[:, None, None, None]
            least = 2.0 ** -39 if max(bt.q_len) * group <= 16 else 2.0 ** -54
            t = t + (2.0 ** -32 * (count @ v.abs())[:, None] + least * count.sum(1)[:, None] * largest) / total
        rows = slice(t0, t0 + n)
        out[rows], tol[rows] = (x.permute(2, 0, 1, 3).reshape(n, bt.heads, bt.dim) for x in (o, t))
    return out, tol
