"""The 8-bit cache's and the window's entry points on the host: workspace sizes and refusals before any CUDA call
(no GPU needed)."""
import ctypes
import math

import pytest

import top_routing_grouped_router_gb300 as moe
from top_routing_grouped_router_gb300 import build as moe_build

FAKE = 1 << 20  # an aligned address that no refused call touches
OK, NULLPTR, SHAPE, DTYPE, WORKSPACE, ALIGN = 0, -1, -2, -3, -4, -5
GOOD = dict(n_tokens=8, n_seqs=4, n_heads=8, n_kv_heads=2, head_dim=64, page_size=32, n_pages=10, max_pages=5, max_q=4,
            act="bf16")


@pytest.fixture(scope="module")
def L():
    moe_build.build()
    return moe.lib()


def _shape(**kw):
    return moe.make_attn_shape(**{**GOOD, **kw})


def _cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, ps=4096, hs=2048, ts=64, sps=4, shs=2, block=16):
    return moe.MoEKVCacheQ8(k, v, ks, vs, ps, hs, ts, sps, shs, block)


CACHE = [(dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(ks=None), NULLPTR), (dict(vs=None), NULLPTR),
         (dict(block=0), SHAPE), (dict(block=-16), SHAPE), (dict(block=24), SHAPE), (dict(block=64), SHAPE),
         (dict(ts=48), SHAPE), (dict(hs=32), SHAPE), (dict(shs=1), SHAPE), (dict(ps=-4096), SHAPE), (dict(sps=-1), SHAPE),
         (dict(ps=(1 << 40) + 16), SHAPE), (dict(ps=4104), ALIGN), (dict(hs=2056), ALIGN), (dict(ts=72), ALIGN),
         (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 4), ALIGN)]
FITS = [dict(ks=FAKE + 1), dict(vs=FAKE + 3), dict(sps=7), dict(block=32), dict(block=1, shs=32)]  # refused later only


def _attend(L, c, shape=None, window=None, **kw):
    a = dict(q=FAKE, qs=512, scale=0.1, out=FAKE, os=512, lse=None, ws=FAKE, need=1 << 40, batch=True)
    a.update(kw)
    s, b = shape or _shape(), moe.MoEAttnBatch(FAKE, FAKE, FAKE)
    return L.moe_paged_attention_q8(ctypes.byref(s), a["q"], a["qs"], None if c is None else ctypes.byref(c),
                                    ctypes.byref(b) if a["batch"] else None, None if window is None else ctypes.byref(window),
                                    a["scale"], a["out"], a["os"], a["lse"], a["ws"], a["need"], None)


def _append(L, c, shape=None, **kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, out=FAKE, os=512, ws=FAKE, need=2048, rot=64, pos=None, batch=True)
    a.update(kw)
    s, b, r = shape or _shape(), moe.MoEAttnBatch(FAKE, FAKE, FAKE), moe.MoERope(a["rot"], 0, 1.0, 1e-6, FAKE, None, None)
    return L.moe_rope_append_q8(ctypes.byref(s), ctypes.byref(r), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                                None if c is None else ctypes.byref(c), ctypes.byref(b) if a["batch"] else None, a["pos"],
                                a["out"], a["os"], a["ws"], a["need"], None)


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_refusals_of_both_calls(L, kw, code):
    assert _attend(L, _cache(**kw)) == code
    assert _append(L, _cache(**kw)) == code


@pytest.mark.parametrize("kw", FITS)
def test_scales_need_no_alignment(L, kw):
    # only the workspace is wrong then
    assert _attend(L, _cache(**kw), need=2047) == WORKSPACE
    assert _append(L, _cache(**kw), need=2047) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=72), SHAPE), (dict(head_dim=60), SHAPE), (dict(page_size=0), SHAPE), (dict(n_kv_heads=3), SHAPE),
    (dict(max_q=9), SHAPE), (dict(n_seqs=0), SHAPE), (dict(act=2), DTYPE)])
def test_shape_refusals(L, kw, code):
    s, n = _shape(**kw), ctypes.c_size_t(0)
    assert L.moe_attn_q8_workspace_size(ctypes.byref(s), 16, ctypes.byref(n)) == code
    assert _attend(L, _cache(ts=128, hs=8192, ps=65536), s, qs=4096, os=4096) == code
    assert _append(L, _cache(ts=128, hs=8192, ps=65536), s, qs=4096, os=4096, ks=4096, vs=4096) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULLPTR), (dict(out=None), NULLPTR), (dict(batch=False), NULLPTR), (dict(scale=math.nan), SHAPE),
    (dict(scale=-math.inf), SHAPE), (dict(qs=504), SHAPE), (dict(os=8), SHAPE), (dict(qs=516), ALIGN), (dict(q=FAKE + 8), ALIGN),
    (dict(out=FAKE + 2), ALIGN), (dict(lse=FAKE + 1), ALIGN), (dict(ws=None), WORKSPACE), (dict(need=2047), WORKSPACE),
    (dict(ws=FAKE + 64), ALIGN)])
def test_attention_refusals(L, kw, code):
    assert _attend(L, _cache(), **kw) == code
    if kw.get("need") != 2047:
        assert _attend(L, _cache(), window=moe.make_attn_window(5, 1), **kw) == code


def test_a_missing_cache_is_refused(L):
    assert _attend(L, None) == NULLPTR and _append(L, None) == NULLPTR


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULLPTR), (dict(k=None), NULLPTR), (dict(v=None), NULLPTR), (dict(out=None), NULLPTR),
    (dict(batch=False), NULLPTR), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(ks=120), SHAPE), (dict(vs=132), ALIGN),
    (dict(k=FAKE + 8), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(need=2047), WORKSPACE)])
def test_append_refusals(L, kw, code):
    assert _append(L, _cache(), **kw) == code


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 3), (5, -1), (-2**31, 0)])
def test_windows_that_are_refused(L, window, sinks):
    s, b, w = _shape(), moe.MoEAttnBatch(FAKE, FAKE, FAKE), moe.make_attn_window(window, sinks)
    assert _attend(L, _cache(), window=w) == SHAPE
    c = moe.MoEKVCache(FAKE, FAKE, 4096, 2048, 64)
    call = lambda w: L.moe_paged_attention_window(ctypes.byref(s), FAKE, 512, ctypes.byref(c), ctypes.byref(b), w, 0.1,  # noqa: E731
                                                  FAKE, 512, None, FAKE, 1 << 30, None)
    assert call(ctypes.byref(w)) == SHAPE
    assert call(None) == NULLPTR


@pytest.mark.parametrize("kw,code", [(dict(k=None), NULLPTR), (dict(ts=56), SHAPE), (dict(q=FAKE + 8), ALIGN),
                                     (dict(need=2047), WORKSPACE), (dict(scale=math.inf), SHAPE)])
def test_window_refusals_are_those_of_attention(L, kw, code):
    a = dict(k=FAKE, ts=64, q=FAKE, need=1 << 30, scale=0.1)
    a.update(kw)
    s, b, w = _shape(), moe.MoEAttnBatch(FAKE, FAKE, FAKE), moe.make_attn_window(5, 1)
    c = moe.MoEKVCache(a["k"], FAKE, 4096, 2048, a["ts"])
    assert L.moe_paged_attention_window(ctypes.byref(s), a["q"], 512, ctypes.byref(c), ctypes.byref(b), ctypes.byref(w),
                                        a["scale"], FAKE, 512, None, FAKE, a["need"], None) == code


def test_workspace_sizes(L):
    n = ctypes.c_size_t(0)
    s = _shape()
    assert L.moe_attn_q8_workspace_size(ctypes.byref(s), 16, None) == NULLPTR
    assert L.moe_attn_q8_workspace_size(None, 16, ctypes.byref(n)) == NULLPTR
    for block in (0, -1, 24, 64):
        assert L.moe_attn_q8_workspace_size(ctypes.byref(s), block, ctypes.byref(n)) == SHAPE
    for kw in (dict(), dict(max_q=1), dict(head_dim=80), dict(act="f32"), dict(n_tokens=500, max_q=300, max_pages=200)):
        for block in (1, 16, 32):
            size = moe.moe_attn_q8_workspace_size(_shape(**kw), block)
            assert size >= 2048
            # the call takes that much, and not a byte less
            s = _shape(**kw)
            wide = 8 * s.head_dim
            c = _cache(ts=s.head_dim, hs=32 * s.head_dim, ps=64 * s.head_dim, shs=32, sps=64, block=block)
            assert _attend(L, c, s, qs=wide, os=wide, need=size - 1) == WORKSPACE


def test_empty_batches_launch_nothing(L):
    s = _shape(n_tokens=0, n_seqs=0, max_q=0)
    r = moe.MoERope(64, 0, 1.0, 0.0, None, None, None)
    w = moe.make_attn_window(1)
    assert L.moe_paged_attention_q8(ctypes.byref(s), None, 0, None, None, None, 0.1, None, 0, None, None, 0, None) == OK
    assert L.moe_paged_attention_window(ctypes.byref(s), None, 0, None, None, ctypes.byref(w), 0.1, None, 0, None, None, 0, None) == OK
    assert L.moe_rope_append_q8(ctypes.byref(s), ctypes.byref(r), None, 0, None, 0, None, 0, None, None, None, None, 0, None,
                                0, None) == OK


def test_binding_of_an_8_bit_cache():
    torch = pytest.importorskip("torch")
    u8 = torch.uint8
    k, s = torch.zeros(10, 2, 32, 64, dtype=u8), torch.zeros(10, 2, 2, dtype=u8)
    c = moe.make_kv_cache_q8(k, k.clone(), s, s.clone())
    assert (c.page_stride, c.head_stride, c.token_stride, c.scale_page_stride, c.scale_head_stride, c.block) == (
        4096, 2048, 64, 4, 2, 16)
    f8 = k.view(torch.float8_e4m3fn)
    assert moe.make_kv_cache_q8(f8, f8, s.view(torch.float8_e8m0fnu), s.view(torch.float8_e8m0fnu)).block == 16
    slots = torch.zeros(10, 32, 2, 64, dtype=u8).transpose(1, 2)
    assert moe.make_kv_cache_q8(slots, slots, s, s).token_stride == 128
    for bad in ((k, k[:9], s, s), (k, slots, s, s), (k.transpose(2, 3), k.transpose(2, 3), s, s), (k.float(), k.float(), s, s),
                (k, k, s.float(), s.float()), (k, k, s, s[:, :1]), (k, k, s[:9], s[:9]), (k, f8, s, s),
                (k, k, torch.zeros(10, 2, 5, dtype=u8), torch.zeros(10, 2, 5, dtype=u8)), (k, k, s[..., :0], s[..., :0]),
                (k, k, s.transpose(1, 2), s.transpose(1, 2).contiguous())):
        with pytest.raises(ValueError):
            moe.make_kv_cache_q8(*bad)


def _on_gpu(t):
    """A host tensor that says it is on the GPU, for calls that are refused before the library."""
    torch = pytest.importorskip("torch")

    class OnGpu(torch.Tensor):
        is_cuda = True

    return t.as_subclass(OnGpu)


def _binding_call(kind=lambda t: t, call="attn", **kw):
    torch = pytest.importorskip("torch")
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    a = dict(q=torch.zeros(8, 8, 64, dtype=bf), k=torch.zeros(8, 2, 64, dtype=bf), v=torch.zeros(8, 2, 64, dtype=bf),
             out=torch.zeros(8, 8, 64, dtype=bf), lse=torch.zeros(8, 8), cu=torch.zeros(5, dtype=i32),
             kv=torch.zeros(4, dtype=i32), table=torch.zeros(4, 5, dtype=i32), cache=torch.zeros(10, 2, 32, 64, dtype=u8),
             scales=torch.zeros(10, 2, 2, dtype=u8), bf_cache=torch.zeros(10, 2, 32, 64, dtype=bf),
             positions=torch.zeros(8, dtype=i32), ws=torch.zeros(1 << 20, dtype=u8))
    a.update(kw)
    a = {n: kind(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    shape, batch = _shape(), moe.make_attn_batch(a["cu"], a["kv"], a["table"])
    if call == "window":
        moe.moe_paged_attention_window(shape, a["q"], moe.make_kv_cache(a["bf_cache"], a["bf_cache"].clone()), batch,
                                       moe.make_attn_window(5), a["out"], lse=a["lse"], workspace=a["ws"], stream=0)
        return
    cache = moe.make_kv_cache_q8(a["cache"], a["cache"], a["scales"], a["scales"])
    if call == "append":
        rope = moe.make_rope(64, device="cpu")
        rope.sizes = None
        moe.moe_rope_append_q8(shape, rope, a["q"], a["k"], a["v"], cache, batch, a["out"], a["positions"], a["ws"], 0)
    else:
        moe.moe_paged_attention_q8(shape, a["q"], cache, batch, a["out"], lse=a["lse"], workspace=a["ws"], stream=0)


WRONG = [("q", lambda t: t.zeros(8, 8, 64)), ("q", lambda t: t.zeros(7, 8, 64).bfloat16()), ("out", lambda t: t.zeros(8, 8, 56).bfloat16()),
         ("cu", lambda t: t.zeros(4).int()), ("kv", lambda t: t.zeros(3).int()), ("table", lambda t: t.zeros(4, 4).int())]


@pytest.mark.parametrize("call,name,make", [(c, n, m) for c in ("attn", "window", "append") for n, m in WRONG] + [
    ("attn", "lse", lambda t: t.zeros(7, 8)), ("window", "lse", lambda t: t.zeros(8, 8).bfloat16()),
    ("attn", "cache", lambda t: t.zeros(9, 2, 32, 64).to(t.uint8)), ("append", "cache", lambda t: t.zeros(10, 2, 32, 80).to(t.uint8)),
    ("window", "bf_cache", lambda t: t.zeros(10, 2, 32, 64)), ("append", "k", lambda t: t.zeros(8, 1, 64).bfloat16()),
    ("append", "v", lambda t: t.zeros(8, 2, 64)), ("append", "positions", lambda t: t.zeros(7).int())])
def test_binding_refuses_wrong_types_and_sizes(call, name, make):
    torch = pytest.importorskip("torch")
    kw = {name: make(torch)}
    if name == "cache" and kw["cache"].shape[0] == 9:
        kw["scales"] = torch.zeros(9, 2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError) as e:
        _binding_call(_on_gpu, call, **kw)
    assert "on the GPU" not in str(e.value)


@pytest.mark.parametrize("call", ["attn", "window", "append"])
def test_binding_refuses_host_tensors(call):
    with pytest.raises(ValueError, match="on the GPU"):
        _binding_call(call=call)
