"""The attention half's entry points on the host: rotation tables against the published
formulas, workspace sizes, and refusals before any CUDA call (no GPU needed)."""
import ctypes
import math

import pytest

import top_routing_grouped_router_gb300 as moe
from top_routing_grouped_router_gb300 import build as moe_build

from attn_ref import rates

FAKE = 1 << 20  # an aligned address that no refused call touches
OK, NULLPTR, SHAPE, DTYPE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


@pytest.mark.parametrize("scaling,factor,trained", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                                    ("yarn", 4.0, 32768), ("yarn", 16.0, 4096)])
@pytest.mark.parametrize("rot", [16, 64, 128, 256])
def test_rope_turns_follow_the_formulas(L, scaling, factor, trained, rot):
    base = 1e6
    turns, mscale = moe.moe_rope_turns(rot, scaling, base, factor, trained)
    f, m = rates(rot, base, scaling, factor, trained)
    assert len(turns) == rot // 2
    assert abs(mscale - m) <= 2.0 ** -24 * m
    for t, x in zip(turns, f):
        # a handful of double-precision roundings, pow and log among them
        assert abs(t / 2.0 ** 64 * 2 * math.pi - x) <= 64 * 2.0 ** -53 * x + 2.0 ** -62


@pytest.mark.parametrize("args", [(0, "none", 1e4, 1.0, 0), (24, "none", 1e4, 1.0, 0), (272, "none", 1e4, 1.0, 0),
                                  (64, 4, 1e4, 1.0, 0), (64, -1, 1e4, 1.0, 0), (64, "none", 1.0, 1.0, 0),
                                  (64, "none", math.nan, 1.0, 0), (64, "linear", 1e4, 0.5, 0),
                                  (64, "ntk", 1e4, math.inf, 0), (64, "yarn", 1e4, 2.0, 0)])
def test_rope_turns_refuses(L, args):
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rope_turns(*args)
    assert e.value.status == SHAPE


GOOD = dict(n_tokens=8, n_seqs=4, n_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_pages=5, max_q=4,
            act="bf16")
BAD_SHAPES = [(dict(n_tokens=-1), SHAPE), (dict(n_tokens=(1 << 20) + 1), SHAPE), (dict(n_seqs=0), SHAPE),
              (dict(n_seqs=(1 << 16) + 1), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_heads=9), SHAPE),
              (dict(n_heads=2048), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(head_dim=60), SHAPE),
              (dict(head_dim=264), SHAPE), (dict(page_size=0), SHAPE), (dict(n_pages=0), SHAPE),
              (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 20, page_size=1 << 12), SHAPE), (dict(max_q=9), SHAPE),
              (dict(max_q=-1), SHAPE), (dict(act=2), DTYPE), (dict(act=7), DTYPE)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_shape_refusals_of_every_call(L, kw, code):
    s = moe.make_attn_shape(**{**GOOD, **kw})
    n = ctypes.c_size_t(0)
    c, b, r = moe.MoEKVCache(FAKE, FAKE, 2048, 1024, 64), moe.MoEAttnBatch(FAKE, FAKE, FAKE), moe.MoERope(
        64, 0, 1.0, 1e-6, FAKE, None, None)
    S, C, B, R = map(ctypes.byref, (s, c, b, r))
    assert L.moe_attn_workspace_size(S, ctypes.byref(n)) == code
    assert L.moe_rope_append(S, R, FAKE, 4096, FAKE, 4096, FAKE, 4096, C, B, None, FAKE, 4096, FAKE, 1 << 30,
                             None) == code
    assert L.moe_paged_attention(S, FAKE, 4096, C, B, 0.1, FAKE, 4096, None, FAKE, 1 << 30, None) == code


def _attn(L, **kw):
    a = dict(q=FAKE, qs=512, k=FAKE, v=FAKE, ps=2048, hs=1024, ts=64, cu=FAKE, kv=FAKE, tb=FAKE, scale=0.1, out=FAKE,
             os=512, lse=None, ws=FAKE, need=1 << 30)
    a.update(kw)
    s = moe.make_attn_shape(**GOOD)
    c, b = moe.MoEKVCache(a["k"], a["v"], a["ps"], a["hs"], a["ts"]), moe.MoEAttnBatch(a["cu"], a["kv"], a["tb"])
    return L.moe_paged_attention(ctypes.byref(s), a["q"], a["qs"], ctypes.byref(c), ctypes.byref(b), a["scale"],
                                 a["out"], a["os"], a["lse"], a["ws"], a["need"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULLPTR), (dict(out=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR),
    (dict(cu=None), NULLPTR), (dict(kv=None), NULLPTR), (dict(tb=None), NULLPTR), (dict(scale=math.nan), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(qs=504), SHAPE), (dict(os=8), SHAPE), (dict(ts=56), SHAPE),
    (dict(hs=32), SHAPE), (dict(ps=-2048), SHAPE), (dict(qs=1 << 31), SHAPE), (dict(os=1 << 40), SHAPE), (dict(qs=516), ALIGN), (dict(os=513), ALIGN), (dict(ps=2052), ALIGN),
    (dict(ts=68), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(out=FAKE + 2), ALIGN), (dict(k=FAKE + 4), ALIGN),
    (dict(v=FAKE + 8), ALIGN), (dict(cu=FAKE + 2), ALIGN), (dict(lse=FAKE + 1), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(need=2047), WORKSPACE), (dict(ws=FAKE + 64), ALIGN)])
def test_attention_refusals(L, kw, code):
    assert _attn(L, **kw) == code


def _rope(L, **kw):
    a = dict(rot=64, ms=1.0, eps=1e-6, turns=FAKE, gq=None, gk=None, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128,
             pos=None, out=FAKE, os=512, ws=FAKE, need=2048)
    a.update(kw)
    s, c, b = moe.make_attn_shape(**GOOD), moe.MoEKVCache(FAKE, FAKE, 2048, 1024, 64), moe.MoEAttnBatch(FAKE, FAKE, FAKE)
    r = moe.MoERope(a["rot"], 0, a["ms"], a["eps"], a["turns"], a["gq"], a["gk"])
    return L.moe_rope_append(ctypes.byref(s), ctypes.byref(r), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                             ctypes.byref(c), ctypes.byref(b), a["pos"], a["out"], a["os"], a["ws"], a["need"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(ms=math.inf), SHAPE),
    (dict(gq=FAKE, eps=-1.0), SHAPE), (dict(gk=FAKE, eps=math.nan), SHAPE), (dict(turns=None), NULLPTR),
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(ks=120), SHAPE), (dict(vs=132), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(gq=FAKE + 8), ALIGN),
    (dict(turns=FAKE + 8), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(need=2047), WORKSPACE)])
def test_rope_refusals(L, kw, code):
    assert _rope(L, **kw) == code


def _q4(L, **kw):
    a = dict(T=4, K=256, N=48, dt="bf16", qb=64, x=FAKE, xs=256, codes=FAKE, scales=FAKE, res=None, rs=0, out=FAKE,
             os=48)
    a.update(kw)
    s = moe.make_q4_linear_shape(a["T"], a["K"], a["N"], a["dt"], a["qb"])
    w = moe.MoEQ4Weight(a["codes"], a["scales"], (ctypes.c_float * 16)())
    return L.moe_q4_linear(ctypes.byref(s), a["x"], a["xs"], ctypes.byref(w), a["res"], a["rs"], a["out"], a["os"],
                           None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 18) + 1), SHAPE), (dict(K=0), SHAPE), (dict(K=252, qb=2), SHAPE),
    (dict(N=0), SHAPE), (dict(qb=0), SHAPE), (dict(qb=33), SHAPE), (dict(qb=96), SHAPE), (dict(dt=2), DTYPE),
    (dict(x=None), NULLPTR), (dict(codes=None), NULLPTR), (dict(scales=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(xs=248), SHAPE), (dict(os=47), SHAPE), (dict(res=FAKE, rs=40), SHAPE), (dict(xs=260), ALIGN),
    (dict(x=FAKE + 8), ALIGN), (dict(codes=FAKE + 4), ALIGN), (dict(scales=FAKE + 2), ALIGN), (dict(out=FAKE + 2), ALIGN),
    (dict(res=FAKE + 2, rs=48), ALIGN)])
def test_q4_linear_refusals(L, kw, code):
    assert _q4(L, **kw) == code


def test_empty_batches_launch_nothing(L):
    # no rows: accepted without a pointer or a GPU
    s = moe.make_attn_shape(**{**GOOD, "n_tokens": 0, "n_seqs": 0, "max_q": 0})
    r = moe.MoERope(64, 0, 1.0, 0.0, None, None, None)
    assert L.moe_paged_attention(ctypes.byref(s), None, 0, None, None, 0.1, None, 0, None, None, 0, None) == OK
    assert L.moe_rope_append(ctypes.byref(s), ctypes.byref(r), None, 0, None, 0, None, 0, None, None, None, None, 0, None,
                             0, None) == OK
    q = moe.make_q4_linear_shape(0, 256, 48)
    assert L.moe_q4_linear(ctypes.byref(q), None, 0, None, None, 0, None, 0, None) == OK


def test_binding_refuses_scattered_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, 64)
    with pytest.raises(ValueError):
        moe._row_stride(x.transpose(1, 2), "q")
    with pytest.raises(ValueError):
        moe._row_stride(x[:, ::2], "q")
    assert moe._row_stride(x.view(4, 512)[:, :256].view(4, 4, 64), "q") == 512
    k = torch.zeros(3, 2, 16, 64)
    with pytest.raises(ValueError):
        moe.make_kv_cache(k, torch.zeros(3, 16, 2, 64).transpose(1, 2))
    with pytest.raises(ValueError):
        moe.make_kv_cache(k.transpose(2, 3), k.transpose(2, 3))
    c = moe.make_kv_cache(torch.zeros(3, 16, 2, 64).transpose(1, 2), torch.zeros(3, 16, 2, 64).transpose(1, 2))
    assert (c.page_stride, c.head_stride, c.token_stride) == (2048, 64, 128)


def _on_gpu(t):
    """A host tensor that says it is on the GPU, for calls that are refused before the library."""
    torch = pytest.importorskip("torch")

    class OnGpu(torch.Tensor):
        is_cuda = True

    return t.as_subclass(OnGpu)


def _binding_call(kind=lambda t: t, **kw):
    """One call of a binding on tensors that are right but for `kw`: name -> tensor."""
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    a = dict(q=torch.zeros(8, 8, 64, dtype=bf), k=torch.zeros(8, 2, 64, dtype=bf), v=torch.zeros(8, 2, 64, dtype=bf),
             out=torch.zeros(8, 8, 64, dtype=bf), lse=torch.zeros(8, 8), cu=torch.zeros(5, dtype=i32),
             kv=torch.zeros(4, dtype=i32), table=torch.zeros(4, 5, dtype=i32), cache=torch.zeros(10, 2, 16, 64, dtype=bf),
             positions=torch.zeros(8, dtype=i32), gamma=torch.ones(64, dtype=bf), x=torch.zeros(4, 256, dtype=bf),
             y=torch.zeros(4, 48, dtype=bf), res=torch.zeros(4, 48, dtype=bf), codes=torch.zeros(48, 128, dtype=torch.uint8),
             scales=torch.zeros(48, 4, dtype=bf), ws=torch.zeros(1 << 20, dtype=torch.uint8), call="attn")
    a.update(kw)
    a = {n: kind(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    if a["call"] == "q4":
        moe.moe_q4_linear(moe.make_q4_linear_shape(4, 256, 48), a["x"], moe.make_q4_weight(a["codes"], a["scales"], [0] * 16),
                          a["y"], residual=a["res"], stream=0)
        return
    shape = moe.make_attn_shape(**GOOD)
    batch, cache = moe.make_attn_batch(a["cu"], a["kv"], a["table"]), moe.make_kv_cache(a["cache"], a["cache"].clone())
    if a["call"] == "rope":
        rope = moe.make_rope(64, q_gamma=a["gamma"], device="cpu")
        rope.sizes = (*rope.sizes[:2], kind is not _on_gpu)  # its table
        moe.moe_rope_append(shape, rope, a["q"], a["k"], a["v"], cache, batch, a["out"], a["positions"], a["ws"], 0)
    else:
        moe.moe_paged_attention(shape, a["q"], cache, batch, a["out"], lse=a["lse"], workspace=a["ws"], stream=0)


@pytest.mark.parametrize("call,name,make", [
    ("attn", "lse", lambda t: t.zeros(8, 8, dtype=t.bfloat16)), ("attn", "lse", lambda t: t.zeros(7, 8)),
    ("attn", "lse", lambda t: t.zeros(8, 7)), ("attn", "q", lambda t: t.zeros(8, 8, 64)),
    ("attn", "q", lambda t: t.zeros(7, 8, 64, dtype=t.bfloat16)), ("attn", "out", lambda t: t.zeros(8, 8, 64).half()),
    ("attn", "out", lambda t: t.zeros(8, 8, 56).bfloat16()), ("attn", "out", lambda t: t.zeros(8, 4, 64).bfloat16()),
    ("attn", "cu", lambda t: t.zeros(5)), ("attn", "cu", lambda t: t.zeros(4).int()), ("attn", "kv", lambda t: t.zeros(3).int()),
    ("attn", "kv", lambda t: t.zeros(4).long()), ("attn", "table", lambda t: t.zeros(4, 4).int()),
    ("attn", "table", lambda t: t.zeros(4, 10).int()[:, ::2]), ("attn", "cache", lambda t: t.zeros(10, 2, 16, 64)),
    ("attn", "cache", lambda t: t.zeros(9, 2, 16, 64).bfloat16()), ("attn", "cache", lambda t: t.zeros(10, 2, 8, 64).bfloat16()),
    ("rope", "k", lambda t: t.zeros(8, 1, 64).bfloat16()), ("rope", "v", lambda t: t.zeros(8, 2, 64)),
    ("rope", "out", lambda t: t.zeros(8, 8, 64)), ("rope", "positions", lambda t: t.zeros(8).long()),
    ("rope", "positions", lambda t: t.zeros(7).int()), ("rope", "gamma", lambda t: t.ones(64)),
    ("rope", "gamma", lambda t: t.ones(60).bfloat16()), ("q4", "x", lambda t: t.zeros(4, 256)),
    ("q4", "x", lambda t: t.zeros(3, 256).bfloat16()), ("q4", "x", lambda t: t.zeros(4, 248).bfloat16()),
    ("q4", "y", lambda t: t.zeros(4, 48)), ("q4", "res", lambda t: t.zeros(4, 48)),
    ("q4", "codes", lambda t: t.zeros(48, 128)), ("q4", "codes", lambda t: t.zeros(47, 128).to(t.uint8)),
    ("q4", "scales", lambda t: t.zeros(48, 4)), ("q4", "scales", lambda t: t.zeros(48, 8).bfloat16())])
def test_binding_refuses_wrong_types_and_sizes(call, name, make):
    # a type, a size or a number of rows that the kernels would read or write past: refused before the library
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError) as e:
        _binding_call(_on_gpu, call=call, **{name: make(torch)})
    assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("call", ["attn", "rope", "q4"])
def test_binding_refuses_host_tensors(call):
    with pytest.raises(ValueError, match="on the GPU"):
        _binding_call(call=call)


def test_binding_takes_any_stride_of_a_single_row():
    # a tensor of one row is contiguous whatever its row stride says
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    x = torch.empty(64, 1, dtype=bf).t()
    assert x.stride() == (1, 1) and moe._row_stride(x, "x") == 64
    q = torch.empty(1, 4, 64, dtype=bf).as_strided((1, 4, 64), (8, 64, 1))
    assert moe._row_stride(q, "q") == 256
    wide = torch.empty(3, 320, dtype=bf)
    assert moe._row_stride(wide[:, :64], "x") == 320 and moe._row_stride(wide[:, 5:6], "x") == 320
    assert moe._row_stride(wide[:, :256].view(3, 4, 64), "q") == 320


def test_binding_follows_a_changed_shape():
    torch = pytest.importorskip("torch")
    s = moe.make_attn_shape(**GOOD)
    assert moe._attn_checks(s)[0] == 8 * 8 * 64 and s._checks[5] is torch.bfloat16
    s.n_tokens, s.dtype = 9, 0
    assert s._checks is None and moe._attn_checks(s)[0] == 9 * 8 * 64 and s._checks[5] is torch.float32
    s = moe.make_q4_linear_shape(4, 256, 48)
    assert moe._q4_checks(s)[:4] == (1024, 192, 256, 48)
    s.T = 5
    assert s._checks is None and moe._q4_checks(s)[:2] == (1280, 240)
