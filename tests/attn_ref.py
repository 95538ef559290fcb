"""The attention half of a layer in 64 bits on the CPU, from the definitions, and the error
bounds of the CUDA kernels' arithmetic (used by the GPU tests)."""
from __future__ import annotations

import dataclasses
import math

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step relative to the value: what rounding to the type costs at most
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
# one fp32 addition or product on the tensor cores (which may truncate) or the CUDA cores
FP32 = 2.0 ** -23


@dataclasses.dataclass
class Batch:
    dtype: str
    heads: int
    kv_heads: int
    dim: int
    page: int
    q_len: list
    kv_len: list
    cu_q: torch.Tensor
    table: torch.Tensor
    pages: int
    q: torch.Tensor        # [tokens][heads][dim]
    k_cache: torch.Tensor  # [pages][kv_heads][page][dim]
    v_cache: torch.Tensor

    @property
    def tokens(self):
        return sum(self.q_len)


def make_batch(dtype, heads, kv_heads, dim, page, q_len, kv_len, seed=0, spread=1.0, fill=float("nan")):
    """A random batch on the CPU; every slot that no sequence holds is `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in kv_len]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(kv_len), max(max(need, default=1), 1)), -7, dtype=torch.int32)
    k, v = (torch.full((pages, kv_heads, page, dim), fill).to(DT[dtype]) for _ in range(2))
    at = 0
    for b, (n, m) in enumerate(zip(need, kv_len)):
        table[b, :n] = order[at:at + n]
        at += n
        for c in (k, v):
            rows = torch.randn(kv_heads, n * page, dim, generator=g).to(DT[dtype])
            rows[:, m:] = fill
            c[table[b, :n].long()] = rows.view(kv_heads, n, page, dim).transpose(0, 1)
    cu = torch.tensor([0] + q_len).cumsum(0).int()
    q = (spread * torch.randn(sum(q_len), heads, dim, generator=g)).to(DT[dtype])
    return Batch(dtype, heads, kv_heads, dim, page, list(q_len), list(kv_len), cu, table, pages, q, k, v)


def keys_of(bt: Batch, b: int, cache):
    """Sequence b's keys (or values) in order: [kv_heads][kv_len][dim], 64 bits."""
    n = -(-bt.kv_len[b] // bt.page)
    pages = bt.table[b, :n].long()
    return cache[pages].transpose(0, 1).reshape(bt.kv_heads, n * bt.page, bt.dim)[:, :bt.kv_len[b]].double()


def attention(bt: Batch, scale):
    """(out, lse, bound on |out - kernel's out|, bound on |lse - kernel's|), 64 bits."""
    out = torch.zeros(bt.tokens, bt.heads, bt.dim, dtype=torch.float64)
    lse = torch.full((bt.tokens, bt.heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    group = bt.heads // bt.kv_heads
    for b, (n, m) in enumerate(zip(bt.q_len, bt.kv_len)):
        if n == 0:
            continue
        t0 = int(bt.cu_q[b])
        k, v = keys_of(bt, b, bt.k_cache), keys_of(bt, b, bt.v_cache)
        for h in range(bt.heads):
            kh, vh = k[h // group], v[h // group]
            q = bt.q[t0:t0 + n, h].double()
            s = q @ kh.T * scale
            hide = torch.arange(m)[None] > torch.arange(m - n, m)[:, None]
            s = s.masked_fill(hide, -math.inf)
            total = torch.logsumexp(s, 1) if m else torch.full((n,), -math.inf, dtype=torch.float64)
            p = torch.nan_to_num(torch.exp(s - total[:, None]), nan=0.0)
            out[t0:t0 + n, h], lse[t0:t0 + n, h] = p @ vh, total
            # a score is off by dim additions of products and a few roundings, relative to the sum of
            # the products' sizes; a probability by twice that, its exponential and its part in a sum
            # of m terms; bf16 rounds the probabilities before the product with v
            size = (q.abs() @ kh.abs().T * abs(scale)).masked_fill(hide, 0).amax(1) if m else torch.zeros(n)
            ds = (bt.dim + 8) * FP32 * size
            dp = 2 * ds + (m + 32) * FP32 + (HALF["bf16"] if bt.dtype == "bf16" else 0)
            tol[t0:t0 + n, h] = dp[:, None] * (p @ vh.abs()) + HALF[bt.dtype] * (p @ vh).abs() + 1e-30
            tol_lse[t0:t0 + n, h] = torch.where(total.isinf(), torch.zeros(()),
                                                ds + (m + 32) * FP32 + 4 * FP32 * total.abs())
    return out, lse, tol, tol_lse


def rates(rot, base, scaling="none", factor=1.0, trained=0):
    """Radians a position of each pair, and the factor on the rotated part (published formulas)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        for i in range(rot // 2):
            r = min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0)
            f[i] = f[i] / factor * r + f[i] * (1 - r)
        return f, 1 + 0.1 * math.log(factor)
    return f, 1.0


def rotate(x, positions, f, mscale, interleaved, gamma=None, eps=1e-6):
    """x [tokens][heads][dim] rotated at `positions`, 64 bits; the norm first if gamma is given."""
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    h = len(f)
    angle = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64))[:, None]
    c, s = mscale * torch.cos(angle), mscale * torch.sin(angle)
    y = x.clone()
    ia = torch.arange(h) * 2 if interleaved else torch.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def q4_dense(codes, scales, codebook, q_block):
    """The weight matrix [N][K] that the codes stand for, 64 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    return torch.tensor(codebook, dtype=torch.float64)[c] * scales.double().repeat_interleave(q_block, 1)
