"""GB300-native sparse Mixture-of-Experts block (Qwen3-MoE style), Python binding.

A thin ctypes binding of the C ABI in ``include/moe.h`` (``libmoe_gb300.so``,
built in-tree by ``top_routing_grouped_router_gb300.build``).  The functions
below keep the C names and only marshal arguments: torch CUDA tensors (or raw
integer device addresses) become pointers, the current torch CUDA stream becomes
the ``stream`` argument.  Every step of the block runs in the library's CUDA
kernels; there is no fallback of any kind, and every call raises if the library
is missing or returns an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "MOE_DT_F32", "MOE_DT_BF16", "MOE_DT_Q4", "MoEError", "MoEShape", "MoEQ4", "lib", "library_path",
    "make_shape", "moe_workspace_size", "moe_route", "moe_permute", "moe_grouped_swiglu", "moe_unpermute",
    "moe_forward", "moe_forward_launches", "moe_read_device_error", "moe_status_string", "EXPORTED_SYMBOLS",
    "moe_forward_static_scratch", "moe_forward_rmsnorm", "moe_forward_lora", "moe_graph_buckets", "moe_graphs_arena_size",
    "DecodeGraphs", "moe_lora_pack_size", "moe_lora_pack", "pack_lora", "moe_static_scratch_read_error",
    "moe_debug_set_waits", "MoEAttnShape", "MoEAttnBatch", "MoEKVCache", "MoERope", "MoEQ4LinearShape", "MoEQ4Weight",
    "make_attn_shape", "make_attn_batch", "make_kv_cache", "make_rope", "make_q4_linear_shape", "make_q4_weight",
    "moe_attn_workspace_size", "moe_rope_turns", "moe_rope_append", "moe_paged_attention", "moe_q4_linear",
    "moe_q4_linear_read_error", "MoEAttnWindow", "MoEKVCacheQ8", "make_attn_window", "make_kv_cache_q8",
    "moe_paged_attention_window", "moe_attn_q8_workspace_size", "moe_rope_append_q8", "moe_paged_attention_q8",
]

MOE_DT_F32, MOE_DT_BF16, MOE_DT_Q4 = 0, 1, 2
_DT = {"f32": MOE_DT_F32, "bf16": MOE_DT_BF16, "q4": MOE_DT_Q4}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmoe_gb300.so")

EXPORTED_SYMBOLS = ("moe_workspace_size", "moe_route", "moe_permute", "moe_grouped_swiglu", "moe_unpermute",
                    "moe_forward", "moe_forward_launches", "moe_read_device_error", "moe_status_string",
                    "moe_forward_static_scratch", "moe_forward_rmsnorm", "moe_forward_lora", "moe_graph_buckets", "moe_graphs_arena_size", "moe_graphs_create",
                    "moe_graphs_bucket", "moe_graphs_run", "moe_graphs_destroy", "moe_lora_pack_size", "moe_lora_pack",
                    "moe_static_scratch_read_error", "moe_debug_set_waits", "moe_attn_workspace_size",
                    "moe_rope_turns", "moe_rope_append", "moe_paged_attention", "moe_q4_linear",
                    "moe_q4_linear_read_error", "moe_paged_attention_window", "moe_attn_q8_workspace_size",
                    "moe_rope_append_q8", "moe_paged_attention_q8")


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {moe_status_string(status)} ({status})")
        self.status = status


class MoEShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("act_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("norm_topk", ctypes.c_int32), ("q_block", ctypes.c_int32)]


class MoELora(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("scale", ctypes.c_float), ("a_gate", ctypes.c_void_p),
                ("b_gate", ctypes.c_void_p), ("a_up", ctypes.c_void_p), ("b_up", ctypes.c_void_p),
                ("a_down", ctypes.c_void_p), ("b_down", ctypes.c_void_p), ("packed", ctypes.c_void_p)]


class MoEQ4(ctypes.Structure):
    _fields_ = [("gate_scales", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
                ("down_scales", ctypes.c_void_p), ("codebook", ctypes.c_float * 16)]


class _Checked(ctypes.Structure):
    _checks = None  # what a call's tensors are held against, made of the fields; a field that is set takes it away

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name != "_checks":
            super().__setattr__("_checks", None)


class MoEAttnShape(_Checked):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_tokens", "n_seqs", "n_heads", "n_kv_heads", "head_dim", "page_size",
                                              "n_pages", "max_pages", "max_q", "dtype")]


class MoEAttnBatch(ctypes.Structure):
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]
    sizes = None  # of make_attn_batch's tensors: sequences that fit, the table's width, whether one is in host memory


class MoEKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]
    sizes = None  # of make_kv_cache's tensors: pages, heads, slots, head size, type, whether one is in host memory


class MoEAttnWindow(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


class MoEKVCacheQ8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride", "scale_page_stride",
                                      "scale_head_stride")] + [("block", ctypes.c_int32)]
    sizes = None  # of make_kv_cache_q8's tensors, as MoEKVCache's


class MoERope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("eps", ctypes.c_float), ("turns", ctypes.c_void_p), ("q_gamma", ctypes.c_void_p),
                ("k_gamma", ctypes.c_void_p)]
    sizes = None  # of make_rope's norm weights: type, length; and whether a tensor is in host memory


class MoEQ4LinearShape(_Checked):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "out_dtype", "q_block")]


class MoEQ4Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("codebook", ctypes.c_float * 16)]
    sizes = None  # of make_q4_weight's tensors: codes, scales, whether one is in host memory


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libmoe_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"CUDA library {library_path} is missing: build it with "
                               f"`python -m top_routing_grouped_router_gb300.build`")
        L = ctypes.CDLL(library_path)
        vp, sz, i32p, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int64
        sp = ctypes.POINTER(MoEShape)
        q4p = ctypes.POINTER(MoEQ4)
        sig = {
            "moe_workspace_size": [sp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_route": [sp, vp, vp, vp, i32p, vp, vp, vp, vp, sz, vp],
            "moe_permute": [sp, i32p, i32p, i32p, i32p, i32p, vp, sz, vp],
            "moe_grouped_swiglu": [sp, vp, i32p, i32p, vp, vp, vp, q4p, vp, vp, sz, vp],
            "moe_unpermute": [sp, vp, vp, i32p, vp, vp],
            "moe_forward": [sp, vp, vp, vp, vp, vp, vp, q4p, vp, i32p, vp, vp, sz, vp],
            "moe_read_device_error": [vp, ctypes.POINTER(ctypes.c_int32), vp],
            "moe_forward_launches": [sp, ctypes.POINTER(ctypes.c_int32)],
            "moe_forward_static_scratch": [sp, vp, vp, vp, vp, vp, vp, q4p, vp, i32p, vp, vp],
            "moe_static_scratch_read_error": [ctypes.POINTER(ctypes.c_int32), vp],
            "moe_debug_set_waits": [ctypes.c_uint64, ctypes.c_int32],
            "moe_forward_rmsnorm": [sp, vp, vp, ctypes.c_float, ctypes.c_int, vp, vp, vp, vp, vp, q4p, vp, vp, i32p,
                                    vp, vp, sz, vp],
            "moe_forward_lora": [sp, vp, vp, vp, vp, vp, vp, q4p, ctypes.POINTER(MoELora), vp, i32p, vp, vp, sz, vp],
            "moe_graph_buckets": [ctypes.c_int, vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int32)],
            "moe_graphs_arena_size": [sp, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
            "moe_graphs_create": [sp, ctypes.c_int, vp, vp, vp, vp, vp, q4p, vp, sz, vp, ctypes.POINTER(vp)],
            "moe_graphs_bucket": [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int32)],
            "moe_graphs_run": [vp, ctypes.c_int, vp, vp, i32p, vp],
            "moe_graphs_destroy": [vp],
            "moe_lora_pack_size": [sp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_lora_pack": [sp, ctypes.POINTER(MoELora), vp, sz, vp],
            "moe_attn_workspace_size": [vp, ctypes.POINTER(ctypes.c_size_t)],
            "moe_rope_turns": [ctypes.c_int32, ctypes.c_int32, ctypes.c_double, ctypes.c_double, ctypes.c_int32, vp,
                               ctypes.POINTER(ctypes.c_float)],
            "moe_rope_append": [vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, sz, vp],
            "moe_paged_attention": [vp, vp, i64, vp, vp, ctypes.c_float, vp, i64, vp, vp, sz, vp],
            "moe_paged_attention_window": [vp, vp, i64, vp, vp, vp, ctypes.c_float, vp, i64, vp, vp, sz, vp],
            "moe_attn_q8_workspace_size": [vp, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
            "moe_rope_append_q8": [vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, sz, vp],
            "moe_paged_attention_q8": [vp, vp, i64, vp, vp, vp, ctypes.c_float, vp, i64, vp, vp, sz, vp],
            "moe_q4_linear": [vp, vp, i64, vp, vp, i64, vp, i64, vp],
            "moe_q4_linear_read_error": [ctypes.POINTER(ctypes.c_int32), vp],
        }
        for name, argtypes in sig.items():
            f = getattr(L, name)
            f.argtypes = argtypes
            f.restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def make_shape(T, H, E, k, I, act="bf16", w="bf16", norm_topk=True, q_block=64) -> MoEShape:
    return MoEShape(int(T), int(H), int(E), int(k), int(I), _DT[act] if isinstance(act, str) else int(act),
                    _DT[w] if isinstance(w, str) else int(w), int(bool(norm_topk)), int(q_block))


def _ptr(t):
    """Device address of a torch tensor, an int address, or None -> NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t):
    return t.numel() * t.element_size()


def _check(rc: int, what: str):
    if rc != 0:
        raise MoEError(rc, what)


def moe_workspace_size(shape: MoEShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_route(shape, x, w_router, b_router, expert_ids, weights, tie_margin=None, logits=None, workspace=None,
              stream=None):
    _check(lib().moe_route(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(b_router), _ptr(expert_ids),
                           _ptr(weights), _ptr(tie_margin), _ptr(logits), _ptr(workspace), _nbytes(workspace),
                           _stream(stream)), "moe_route")


def moe_permute(shape, expert_ids, counts, offsets, order, pos, workspace, stream=None):
    _check(lib().moe_permute(ctypes.byref(shape), _ptr(expert_ids), _ptr(counts), _ptr(offsets), _ptr(order),
                             _ptr(pos), _ptr(workspace), _nbytes(workspace), _stream(stream)), "moe_permute")


def moe_grouped_swiglu(shape, x, offsets, order, w_gate, w_up, w_down, q4, y, workspace, stream=None):
    _check(lib().moe_grouped_swiglu(ctypes.byref(shape), _ptr(x), _ptr(offsets), _ptr(order), _ptr(w_gate),
                                    _ptr(w_up), _ptr(w_down), ctypes.byref(q4) if q4 is not None else None,
                                    _ptr(y), _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "moe_grouped_swiglu")


def moe_unpermute(shape, y, weights, pos, out, stream=None):
    _check(lib().moe_unpermute(ctypes.byref(shape), _ptr(y), _ptr(weights), _ptr(pos), _ptr(out),
                               _stream(stream)), "moe_unpermute")


def moe_forward(shape, x, w_router, b_router, w_gate, w_up, w_down, q4, out, expert_ids_out=None,
                weights_out=None, workspace=None, stream=None):
    _check(lib().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(b_router), _ptr(w_gate),
                             _ptr(w_up), _ptr(w_down), ctypes.byref(q4) if q4 is not None else None, _ptr(out),
                             _ptr(expert_ids_out), _ptr(weights_out), _ptr(workspace), _nbytes(workspace),
                             _stream(stream)), "moe_forward")


def moe_forward_static_scratch(shape, x, w_router, b_router, w_gate, w_up, w_down, q4, out, expert_ids_out=None,
                               weights_out=None, stream=None):
    """moe_forward with the library's fixed 32 MiB device scratch instead of a caller workspace."""
    _check(lib().moe_forward_static_scratch(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(b_router),
                                            _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                            ctypes.byref(q4) if q4 is not None else None, _ptr(out),
                                            _ptr(expert_ids_out), _ptr(weights_out), _stream(stream)),
           "moe_forward_static_scratch")


def moe_debug_set_waits(limit_ns: int = 2_000_000_000, extra_need: int = 0):
    """Failure-path test hook: the bounded device waits' limit and an unreachable extra count
    for the down tiles' h wait (see moe.h).  Call with no arguments to restore the defaults."""
    _check(lib().moe_debug_set_waits(int(limit_ns), int(extra_need)), "moe_debug_set_waits")


def moe_static_scratch_read_error(stream=None) -> int:
    """Reads and clears the device error word of the static scratch array (synchronises the stream)."""
    code = ctypes.c_int32(0)
    _check(lib().moe_static_scratch_read_error(ctypes.byref(code), _stream(stream)),
           "moe_static_scratch_read_error")
    return code.value


def moe_forward_rmsnorm(shape, hs, gamma, eps, w_router, b_router, w_gate, w_up, w_down, q4, out, add_residual=True,
                        x_norm_out=None, expert_ids_out=None, weights_out=None, workspace=None, stream=None):
    """out = hs + MoE(RMSNorm(hs) * gamma) (the residual only with add_residual)."""
    _check(lib().moe_forward_rmsnorm(ctypes.byref(shape), _ptr(hs), _ptr(gamma), float(eps), int(bool(add_residual)),
                                     _ptr(w_router), _ptr(b_router), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                     ctypes.byref(q4) if q4 is not None else None, _ptr(out), _ptr(x_norm_out),
                                     _ptr(expert_ids_out), _ptr(weights_out), _ptr(workspace), _nbytes(workspace),
                                     _stream(stream)), "moe_forward_rmsnorm")


def make_lora(rank, scale, a_gate, b_gate, a_up, b_up, a_down, b_down, packed=None) -> MoELora:
    """The moe_lora struct over device tensors (fp32, row-major; see moe.h for the shapes);
    `packed` is a buffer written by moe_lora_pack / pack_lora, or None."""
    return MoELora(int(rank), float(scale), _ptr(a_gate), _ptr(b_gate), _ptr(a_up), _ptr(b_up), _ptr(a_down),
                   _ptr(b_down), _ptr(packed))


def moe_lora_pack_size(shape: MoEShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_lora_pack_size(ctypes.byref(shape), ctypes.byref(n)), "moe_lora_pack_size")
    return n.value


def moe_lora_pack(shape: MoEShape, lora: MoELora, packed, stream=None):
    """Packs the adapters of `lora` into the device buffer `packed` (moe_lora_pack_size bytes)."""
    _check(lib().moe_lora_pack(ctypes.byref(shape), ctypes.byref(lora), _ptr(packed), _nbytes(packed),
                               _stream(stream)), "moe_lora_pack")


def pack_lora(shape: MoEShape, lora: MoELora, device=None, stream=None) -> MoELora:
    """A copy of `lora` that carries a freshly written pack.  The pack is a uint8 tensor on
    `device`, kept alive as the returned struct's `pack_tensor` attribute."""
    import torch
    buf = torch.empty(moe_lora_pack_size(shape), dtype=torch.uint8, device=device or "cuda")
    moe_lora_pack(shape, lora, buf, stream)
    out = MoELora(lora.rank, lora.scale, lora.a_gate, lora.b_gate, lora.a_up, lora.b_up, lora.a_down, lora.b_down,
                  _ptr(buf))
    out.pack_tensor = buf
    return out


def moe_forward_lora(shape, x, w_router, b_router, w_gate, w_up, w_down, q4, lora: MoELora, out, expert_ids_out=None,
                     weights_out=None, workspace=None, stream=None):
    """moe_forward with LoRA adapters on the expert projections."""
    _check(lib().moe_forward_lora(ctypes.byref(shape), _ptr(x), _ptr(w_router), _ptr(b_router), _ptr(w_gate),
                                  _ptr(w_up), _ptr(w_down), ctypes.byref(q4) if q4 is not None else None,
                                  ctypes.byref(lora), _ptr(out), _ptr(expert_ids_out), _ptr(weights_out),
                                  _ptr(workspace), _nbytes(workspace), _stream(stream)), "moe_forward_lora")


def moe_forward_launches(shape: MoEShape) -> int:
    n = ctypes.c_int32(0)
    _check(lib().moe_forward_launches(ctypes.byref(shape), ctypes.byref(n)), "moe_forward_launches")
    return n.value


def moe_read_device_error(workspace, stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(lib().moe_read_device_error(_ptr(workspace), ctypes.byref(code), _stream(stream)),
           "moe_read_device_error")
    return code.value


def moe_graph_buckets(max_bs: int) -> list:
    """Batch-size buckets of the decode graphs for max_bs (host only)."""
    buf = (ctypes.c_int32 * 64)()
    n = ctypes.c_int32(0)
    _check(lib().moe_graph_buckets(int(max_bs), ctypes.cast(buf, ctypes.c_void_p), 64, ctypes.byref(n)),
           "moe_graph_buckets")
    return list(buf[:n.value])


def moe_graphs_arena_size(shape: MoEShape, max_bs: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_graphs_arena_size(ctypes.byref(shape), int(max_bs), ctypes.byref(n)), "moe_graphs_arena_size")
    return n.value


class DecodeGraphs:
    """Bucketed CUDA-graph decode around moe_forward (moe_graphs_* of the C ABI).

    The arena (a device uint8 tensor of moe_graphs_arena_size bytes) is allocated here and
    kept alive with the graphs; the weights are captured by address and must outlive them.
    """

    def __init__(self, shape: MoEShape, max_bs: int, w_router, b_router, w_gate, w_up, w_down, q4=None,
                 device=None, stream=None):
        import torch
        self.shape = shape
        if device is None:
            device = w_router.device if hasattr(w_router, "device") else torch.device("cuda")
        self.arena = torch.zeros(moe_graphs_arena_size(shape, max_bs), dtype=torch.uint8, device=device)
        self._keep = (w_router, b_router, w_gate, w_up, w_down, q4)
        self._stream = stream if stream is not None else torch.cuda.Stream(device=self.arena.device)
        h = ctypes.c_void_p(0)
        _check(lib().moe_graphs_create(ctypes.byref(shape), int(max_bs), _ptr(w_router), _ptr(b_router),
                                       _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                       ctypes.byref(q4) if q4 is not None else None, _ptr(self.arena),
                                       self.arena.numel(), _stream(self._stream), ctypes.byref(h)),
               "moe_graphs_create")
        self._h = h
        self.buckets = moe_graph_buckets(max_bs)

    def bucket(self, T: int) -> int:
        b = ctypes.c_int32(0)
        _check(lib().moe_graphs_bucket(self._h, int(T), ctypes.byref(b)), "moe_graphs_bucket")
        return b.value

    def run(self, T: int, x, out, expert_ids_out=None, stream=None):
        """One decode step of T tokens: x [T][H] in, out [T][H] out (device or host tensors)."""
        st = self._stream if stream is None else stream
        _check(lib().moe_graphs_run(self._h, int(T), _ptr(x), _ptr(out), _ptr(expert_ids_out), _stream(st)),
               "moe_graphs_run")

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().moe_graphs_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- the attention half of a decoder layer ----------------------------------------------

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def make_attn_shape(n_tokens, n_seqs, n_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, max_q,
                    act="bf16") -> MoEAttnShape:
    return MoEAttnShape(int(n_tokens), int(n_seqs), int(n_heads), int(n_kv_heads), int(head_dim), int(page_size),
                        int(n_pages), int(max_pages), int(max_q), _DT[act] if isinstance(act, str) else int(act))


_INT32 = -1  # of _torch_dtype only


def _torch_dtype(code):
    """The torch type of MOE_DT_F32, MOE_DT_BF16 or _INT32 (None of any other)."""
    global _torch_dtype
    import torch
    _torch_dtype = {MOE_DT_F32: torch.float32, MOE_DT_BF16: torch.bfloat16, _INT32: torch.int32}.get
    return _torch_dtype(code)


def _need(t, what, dtypes):
    """A contiguous tensor of one of these types (an int address or None is the caller's own matter); whether it is in
    host memory, which the call that uses it refuses."""
    if t is None or isinstance(t, int):
        return False
    if str(t.dtype)[6:] not in dtypes or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {' or '.join(dtypes)} tensor, not {t.dtype} with strides {t.stride()}")
    return not t.is_cuda


def make_attn_batch(cu_q, kv_len, block_table) -> MoEAttnBatch:
    """The sequences of a batch: int32 device tensors cu_q [B + 1], kv_len [B], block_table [B][max_pages]."""
    named = (cu_q, "cu_q"), (kv_len, "kv_len"), (block_table, "block_table")
    host = [_need(t, what, ("int32",)) for t, what in named]
    out = MoEAttnBatch(_ptr(cu_q), _ptr(kv_len), _ptr(block_table))
    out.tensors = (cu_q, kv_len, block_table)
    if not any(isinstance(t, int) for t in out.tensors):
        out.sizes = min(len(cu_q) - 1, len(kv_len), len(block_table)), block_table.shape[1], any(host)
    return out


def make_kv_cache(k, v) -> MoEKVCache:
    """A paged cache over device tensors k, v of logical shape [pages][kv heads][slots][head dim]: any strides (the
    same for both) whose last is 1, so a [pages][slots][heads][dim] cache is passed as its transpose(1, 2)."""
    if k.stride() != v.stride() or k.shape != v.shape or k.stride(3) != 1 or k.dtype != v.dtype:
        raise ValueError("k and v need equal shapes, strides and types, and contiguous head elements")
    out = MoEKVCache(_ptr(k), _ptr(v), k.stride(0), k.stride(1), k.stride(2))
    out.tensors = (k, v)
    out.sizes = (*k.shape, k.dtype, not (k.is_cuda and v.is_cuda))
    return out


def make_kv_cache_q8(k, v, k_scale, v_scale) -> MoEKVCacheQ8:
    """A paged cache in 8 bits: codes k, v (uint8 or float8_e4m3fn) of logical shape [pages][kv heads][slots][head dim]
    with strides as in make_kv_cache, and the blocks' powers of two k_scale, v_scale (uint8 or float8_e8m0fnu) of
    logical shape [pages][kv heads][slots / block], whose last stride is 1."""
    if k.stride() != v.stride() or k.shape != v.shape or k.stride(3) != 1 or k.dtype != v.dtype:
        raise ValueError("k and v need equal shapes, strides and types, and contiguous head elements")
    if (k_scale.shape != v_scale.shape or k_scale.stride() != v_scale.stride() or k_scale.dtype != v_scale.dtype or
            k_scale.dim() != 3 or (k_scale.stride(2) != 1 and k_scale.shape[2] != 1)):
        raise ValueError("k_scale and v_scale need equal shapes [pages, heads, blocks], strides and types, and contiguous blocks")
    if str(k.dtype)[6:] not in ("uint8", "float8_e4m3fn") or str(k_scale.dtype)[6:] not in ("uint8", "float8_e8m0fnu"):
        raise ValueError(f"codes are uint8 or float8_e4m3fn, scales uint8 or float8_e8m0fnu, not {k.dtype}, {k_scale.dtype}")
    blocks = k_scale.shape[2]
    if k_scale.shape[:2] != k.shape[:2] or blocks == 0 or k.shape[2] % blocks:
        raise ValueError(f"scales {list(k_scale.shape)} do not divide the slots of a cache {list(k.shape)}")
    out = MoEKVCacheQ8(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), k.stride(0), k.stride(1), k.stride(2),
                       k_scale.stride(0), k_scale.stride(1), k.shape[2] // blocks)
    out.tensors = (k, v, k_scale, v_scale)
    out.sizes = (*k.shape, "8-bit", not all(t.is_cuda for t in out.tensors))
    return out


def make_attn_window(window, sinks=0) -> MoEAttnWindow:
    """A token sees the `window` keys up to its own, and the sequence's first `sinks` keys."""
    fit = lambda x: max(-1, min(int(x), (1 << 31) - 1))  # noqa: E731 -- no sequence is longer; below 0 stays refused
    return MoEAttnWindow(fit(window), fit(sinks))


def moe_rope_turns(rot_dim, scaling="none", base=10000.0, factor=1.0, trained_len=0):
    """(turns, mscale): the rotation table as a list of rot_dim / 2 integers in units of 2^-64 turn (host only)."""
    turns = (ctypes.c_uint64 * max(1, int(rot_dim) // 2))()
    mscale = ctypes.c_float(0)
    _check(lib().moe_rope_turns(int(rot_dim), _SCALING[scaling] if isinstance(scaling, str) else int(scaling),
                                float(base), float(factor), int(trained_len), turns, ctypes.byref(mscale)),
           "moe_rope_turns")
    return list(turns), mscale.value


def make_rope(rot_dim, base=10000.0, interleaved=False, scaling="none", factor=1.0, trained_len=0, q_gamma=None,
              k_gamma=None, eps=1e-6, device=None) -> MoERope:
    """The moe_rope struct with its table on `device`; q_gamma / k_gamma are the optional head norms' weights.  The
    struct keeps the table and the weights alive."""
    import torch
    turns, mscale = moe_rope_turns(rot_dim, scaling, base, factor, trained_len)
    table = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device or "cuda")
    out = MoERope(int(rot_dim), int(bool(interleaved)), mscale, float(eps), _ptr(table), _ptr(q_gamma),
                  _ptr(k_gamma))
    out.tensors = (table, q_gamma, k_gamma)
    gammas = (q_gamma, "q_gamma"), (k_gamma, "k_gamma")
    on_host = any([_need(t, what, ("float32", "bfloat16")) for t, what in gammas]) or not table.is_cuda
    known = {(t.dtype, t.numel()) for t, _ in gammas if t is not None and not isinstance(t, int)}
    if len(known) > 1:
        raise ValueError(f"q_gamma and k_gamma differ: {known}")
    if known or on_host:
        out.sizes = (*(known.pop() if known else (None, None)), on_host)
    return out


def make_q4_linear_shape(T, K, N, out="bf16", q_block=64) -> MoEQ4LinearShape:
    return MoEQ4LinearShape(int(T), int(K), int(N), _DT[out] if isinstance(out, str) else int(out), int(q_block))


def make_q4_weight(codes, scales, codebook) -> MoEQ4Weight:
    """One 4-bit weight matrix: codes [N][K/2] uint8, scales [N][K/q_block] bf16, 16 codebook values (host)."""
    host = _need(codes, "codes", ("uint8",)), _need(scales, "scales", ("bfloat16",))
    out = MoEQ4Weight(_ptr(codes), _ptr(scales), (ctypes.c_float * 16)(*[float(c) for c in codebook]))
    out.tensors = (codes, scales)
    if not any(isinstance(t, int) for t in out.tensors):
        out.sizes = codes.numel(), scales.numel(), any(host)
    return out


def _row_stride(t, what):
    """Elements between the rows of a [rows][heads][dim] or [rows][cols] tensor whose rows are contiguous."""
    st = t.stride()
    if (st[-1] != 1 and t.shape[-1] != 1) or (len(st) == 3 and st[1] != t.shape[2] and t.shape[1] != 1):
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return st[0] if t.shape[0] != 1 else t.numel()  # a single row's own stride says nothing


def _wrong(*tensors):
    """The error of the first (name, tensor, type, sizes) whose tensor is not that; its rows may be more."""
    for what, t, dtype, (rows, *sizes) in tensors:
        if t is not None and (t.dtype is not dtype or t.shape[0] < rows or list(t.shape[1:]) != sizes):
            return ValueError(f"{what}: {dtype} {[rows, *sizes]} (more rows are fine), not {t.dtype} {list(t.shape)}")
    for what, t, *_ in tensors:
        if t is not None and not t.is_cuda:
            return ValueError(f"{what}: not on the GPU")
    return ValueError("a tensor's type, size or device is wrong")


def _attn_checks(shape):
    """What the tensors of a call are held against: elements of q and k, their rows' widths, the type, the sizes of the
    batch's, the cache's and the rotation's tensors, the type of positions, and the sizes of an 8-bit cache."""
    n, dtype = shape.n_tokens, _torch_dtype(shape.dtype)
    wide, kv_wide = shape.n_heads * shape.head_dim, shape.n_kv_heads * shape.head_dim
    shape._checks = (n * wide, n * kv_wide, wide, kv_wide, shape.head_dim, dtype, (shape.n_seqs, shape.max_pages, False),
                     (shape.n_pages, shape.n_kv_heads, shape.page_size, shape.head_dim, dtype, False),
                     (dtype, shape.head_dim, False), _torch_dtype(_INT32),
                     (shape.n_pages, shape.n_kv_heads, shape.page_size, shape.head_dim, "8-bit", False))
    return shape._checks


def _q4_checks(shape):
    """The same of a 4-bit linear: elements of x and out, a row's of each, their types, and the weight's sizes."""
    T, K, N, q_block = shape.T, shape.K, shape.N, shape.q_block
    shape._checks = (T * K, T * N, K, N, _torch_dtype(MOE_DT_BF16), _torch_dtype(shape.out_dtype),
                     (N * K // 2, N * K // q_block if q_block > 0 else 0, False))
    return shape._checks


def _check_rope(rope, sizes):
    """That the rotation's norm weights have this type and length, and that its tensors are on the GPU."""
    if rope.sizes[0] is not None and rope.sizes[:2] != sizes[:2]:
        raise ValueError(f"q_gamma, k_gamma: {sizes[0]} [{sizes[1]}], not {rope.sizes[0]} [{rope.sizes[1]}]")
    if rope.sizes[2]:
        raise ValueError("rope: not on the GPU")


def _check_batch(batch, cache, batch_sizes, cache_sizes):
    """That the tensors of the batch and of the cache have these sizes; more sequences and pages are fine."""
    if batch.sizes is not None:
        if batch.sizes[0] < batch_sizes[0] or batch.sizes[1] != batch_sizes[1]:
            raise ValueError("batch: tensors for %d sequences of %d pages, not %d of %d" %
                             (*batch.sizes[:2], *batch_sizes[:2]))
        if batch.sizes[2]:
            raise ValueError("batch: not on the GPU")
    if cache.sizes is None:  # put together by hand: the library reads as much as its own kind of cache holds
        kind = MoEKVCacheQ8 if cache_sizes[4] == "8-bit" else MoEKVCache
        if not isinstance(cache, kind):
            raise ValueError(f"cache: a {kind.__name__}, not a {type(cache).__name__}")
    else:
        if cache.sizes[0] < cache_sizes[0] or cache.sizes[1:5] != cache_sizes[1:5]:
            raise ValueError(f"cache: {cache.sizes[4]} {cache.sizes[:4]}, not {cache_sizes[4]} {cache_sizes[:4]}")
        if cache.sizes[5]:
            raise ValueError("cache: not on the GPU")


def _current_stream():
    """The raw handle of torch's current stream on the current device."""
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    _current_stream = lambda: raw(device())  # noqa: E731 -- a fraction of a microsecond; the Stream object costs several
    return _current_stream()


def moe_attn_workspace_size(shape: MoEAttnShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_attn_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "moe_attn_workspace_size")
    return n.value


# These calls are made several times a layer and step: structs pass by their addresses, nothing is looked up twice
# and the tensors are checked in one expression, so that the host keeps ahead of kernels of a few microseconds.

def moe_rope_append(shape, rope, q, k, v, cache, batch, q_out, positions=None, workspace=None, stream=None):
    """q_out = rotated q; rotated k and v into their cache slots.  q, q_out [N][heads][dim], k, v [N][kv heads][dim]
    (rows may be slices of a wider tensor), positions int32 [N]."""
    at = ctypes.addressof
    (need, kv_need, wide, kv_wide, dim, dtype, batch_sizes, cache_sizes, rope_sizes, int32,
     _) = shape._checks or _attn_checks(shape)
    if batch.sizes != batch_sizes or cache.sizes != cache_sizes:
        _check_batch(batch, cache, batch_sizes, cache_sizes)
    if rope.sizes is not None and rope.sizes != rope_sizes:
        _check_rope(rope, rope_sizes)
    if (q.dtype is not dtype or k.dtype is not dtype or v.dtype is not dtype or q_out.dtype is not dtype or
            q.numel() < need or k.numel() < kv_need or v.numel() < kv_need or q_out.numel() < need or
            not (q.is_cuda and k.is_cuda and v.is_cuda and q_out.is_cuda)):
        n, heads, kv_heads = shape.n_tokens, shape.n_heads, shape.n_kv_heads
        raise _wrong(("q", q, dtype, (n, heads, dim)), ("k", k, dtype, (n, kv_heads, dim)),
                     ("v", v, dtype, (n, kv_heads, dim)), ("q_out", q_out, dtype, (n, heads, dim)))
    if positions is not None and type(positions) is not int:
        if (positions.dtype is not int32 or positions.numel() * wide < need or not positions.is_contiguous() or
                not positions.is_cuda):
            raise _wrong(("positions (contiguous)", positions, int32, (shape.n_tokens,)))
        positions = positions.data_ptr()
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace: not on the GPU")
    # elements between rows; heads that follow one another in rows far enough apart need no second look
    q_row, head, elem = q.stride()
    if head != dim or elem != 1 or q_row < wide:
        q_row = _row_stride(q, "q")
    k_row, head, elem = k.stride()
    if head != dim or elem != 1 or k_row < kv_wide:
        k_row = _row_stride(k, "k")
    v_row, head, elem = v.stride()
    if head != dim or elem != 1 or v_row < kv_wide:
        v_row = _row_stride(v, "v")
    out_row, head, elem = q_out.stride()
    if head != dim or elem != 1 or out_row < wide:
        out_row = _row_stride(q_out, "q_out")
    rc = (_lib or lib()).moe_rope_append(
        at(shape), at(rope), q.data_ptr(), q_row, k.data_ptr(), k_row, v.data_ptr(), v_row, at(cache), at(batch), positions,
        q_out.data_ptr(), out_row, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.nbytes, _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "moe_rope_append")


def moe_paged_attention(shape, q, cache, batch, out, scale=None, lse=None, workspace=None, stream=None):
    """Causal attention of the new tokens' q over the paged cache; scale defaults to head_dim ** -0.5.  q, out
    [N][heads][dim] (rows may be slices of a wider tensor), lse fp32 [N][heads]."""
    at = ctypes.addressof
    need, _, wide, _, dim, dtype, batch_sizes, cache_sizes, _, _, _ = shape._checks or _attn_checks(shape)
    if batch.sizes != batch_sizes or cache.sizes != cache_sizes:
        _check_batch(batch, cache, batch_sizes, cache_sizes)
    if (q.dtype is not dtype or out.dtype is not dtype or q.numel() < need or out.numel() < need or
            not (q.is_cuda and out.is_cuda)):
        sizes = shape.n_tokens, shape.n_heads, dim
        raise _wrong(("q", q, dtype, sizes), ("out", out, dtype, sizes))
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace: not on the GPU")
    if lse is not None:
        fp32 = _torch_dtype(MOE_DT_F32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        if lse.dtype is not fp32 or lse.numel() * dim < need or not lse.is_cuda:
            raise _wrong(("lse", lse, fp32, (shape.n_tokens, shape.n_heads)))
        lse = lse.data_ptr()
    q_row, head, elem = q.stride()
    if head != dim or elem != 1 or q_row < wide:
        q_row = _row_stride(q, "q")
    out_row, head, elem = out.stride()
    if head != dim or elem != 1 or out_row < wide:
        out_row = _row_stride(out, "out")
    rc = (_lib or lib()).moe_paged_attention(
        at(shape), q.data_ptr(), q_row, at(cache), at(batch), dim ** -0.5 if scale is None else scale, out.data_ptr(),
        out_row, lse, None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "moe_paged_attention")


def moe_attn_q8_workspace_size(shape: MoEAttnShape, block: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_attn_q8_workspace_size(ctypes.byref(shape), int(block), ctypes.byref(n)), "moe_attn_q8_workspace_size")
    return n.value


def _head_rows(t, what, dim, wide):
    """Elements between the rows of [rows][heads][dim] whose heads follow one another."""
    row, head, elem = t.stride()
    return row if head == dim and elem == 1 and row >= wide else _row_stride(t, what)


def moe_rope_append_q8(shape, rope, q, k, v, cache, batch, q_out, positions=None, workspace=None, stream=None):
    """moe_rope_append into an 8-bit cache (make_kv_cache_q8)."""
    at = ctypes.addressof
    (need, kv_need, wide, kv_wide, dim, dtype, batch_sizes, _, rope_sizes, int32,
     cache_sizes) = shape._checks or _attn_checks(shape)
    if batch.sizes != batch_sizes or cache.sizes != cache_sizes:
        _check_batch(batch, cache, batch_sizes, cache_sizes)
    if rope.sizes is not None and rope.sizes != rope_sizes:
        _check_rope(rope, rope_sizes)
    if (q.dtype is not dtype or k.dtype is not dtype or v.dtype is not dtype or q_out.dtype is not dtype or
            q.numel() < need or k.numel() < kv_need or v.numel() < kv_need or q_out.numel() < need or
            not (q.is_cuda and k.is_cuda and v.is_cuda and q_out.is_cuda)):
        n, heads, kv_heads = shape.n_tokens, shape.n_heads, shape.n_kv_heads
        raise _wrong(("q", q, dtype, (n, heads, dim)), ("k", k, dtype, (n, kv_heads, dim)),
                     ("v", v, dtype, (n, kv_heads, dim)), ("q_out", q_out, dtype, (n, heads, dim)))
    if positions is not None and type(positions) is not int:
        if (positions.dtype is not int32 or positions.numel() * wide < need or not positions.is_contiguous() or
                not positions.is_cuda):
            raise _wrong(("positions (contiguous)", positions, int32, (shape.n_tokens,)))
        positions = positions.data_ptr()
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace: not on the GPU")
    rc = (_lib or lib()).moe_rope_append_q8(
        at(shape), at(rope), q.data_ptr(), _head_rows(q, "q", dim, wide), k.data_ptr(), _head_rows(k, "k", dim, kv_wide),
        v.data_ptr(), _head_rows(v, "v", dim, kv_wide), at(cache), at(batch), positions, q_out.data_ptr(),
        _head_rows(q_out, "q_out", dim, wide), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.nbytes, _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "moe_rope_append_q8")


def _attend(name, shape, q, cache, cache_sizes, batch, window, out, scale, lse, workspace, stream):
    """What moe_paged_attention_window and moe_paged_attention_q8 share: the checks of moe_paged_attention, and the call."""
    at = ctypes.addressof
    need, _, wide, _, dim, dtype, batch_sizes, _, _, _, _ = shape._checks
    if batch.sizes != batch_sizes or cache.sizes != cache_sizes:
        _check_batch(batch, cache, batch_sizes, cache_sizes)
    if (q.dtype is not dtype or out.dtype is not dtype or q.numel() < need or out.numel() < need or
            not (q.is_cuda and out.is_cuda)):
        sizes = shape.n_tokens, shape.n_heads, dim
        raise _wrong(("q", q, dtype, sizes), ("out", out, dtype, sizes))
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace: not on the GPU")
    if lse is not None:
        fp32 = _torch_dtype(MOE_DT_F32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        if lse.dtype is not fp32 or lse.numel() * dim < need or not lse.is_cuda:
            raise _wrong(("lse", lse, fp32, (shape.n_tokens, shape.n_heads)))
        lse = lse.data_ptr()
    rc = getattr(_lib or lib(), name)(
        at(shape), q.data_ptr(), _head_rows(q, "q", dim, wide), at(cache), at(batch), None if window is None else at(window),
        dim ** -0.5 if scale is None else scale, out.data_ptr(), _head_rows(out, "out", dim, wide), lse,
        None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, name)


def moe_paged_attention_window(shape, q, cache, batch, window, out, scale=None, lse=None, workspace=None, stream=None):
    """moe_paged_attention where a token sees the keys of its window and the sequence's first keys (make_attn_window)."""
    _attend("moe_paged_attention_window", shape, q, cache, (shape._checks or _attn_checks(shape))[7], batch, window, out, scale,
            lse, workspace, stream)


def moe_paged_attention_q8(shape, q, cache, batch, out, window=None, scale=None, lse=None, workspace=None, stream=None):
    """moe_paged_attention over an 8-bit cache (make_kv_cache_q8), over all keys or with a window (make_attn_window)."""
    _attend("moe_paged_attention_q8", shape, q, cache, (shape._checks or _attn_checks(shape))[10], batch, window, out, scale,
            lse, workspace, stream)


def moe_q4_linear(shape, x, weight, out, residual=None, stream=None):
    """out = x . W^T (+ residual) with a 4-bit weight (make_q4_weight); x [T][K] and residual [T][N] bf16, out [T][N]."""
    at = ctypes.addressof
    need, out_need, K, N, bf16, out_dtype, sizes = shape._checks or _q4_checks(shape)
    if weight.sizes is not None and weight.sizes != sizes:
        raise ValueError("weight: (bytes of codes, scales, in host memory) %s, not %s" % (weight.sizes, sizes) if
                         weight.sizes[:2] != sizes[:2] else "weight: not on the GPU")
    if (x.dtype is not bf16 or out.dtype is not out_dtype or x.numel() < need or out.numel() < out_need or
            not (x.is_cuda and out.is_cuda)):
        raise _wrong(("x", x, bf16, (shape.T, K)), ("out", out, out_dtype, (shape.T, N)))
    res_row = 0
    if residual is not None:
        if residual.dtype is not bf16 or residual.numel() < out_need or not residual.is_cuda:
            raise _wrong(("residual", residual, bf16, (shape.T, N)))
        res_row, elem = residual.stride()
        if elem != 1 or res_row < N:
            res_row = _row_stride(residual, "residual")
        residual = residual.data_ptr()
    x_row, elem = x.stride()
    if elem != 1 or x_row < K:
        x_row = _row_stride(x, "x")
    out_row, elem = out.stride()
    if elem != 1 or out_row < N:
        out_row = _row_stride(out, "out")
    rc = (_lib or lib()).moe_q4_linear(at(shape), x.data_ptr(), x_row, at(weight), residual, res_row, out.data_ptr(), out_row,
                                       _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "moe_q4_linear")


def moe_q4_linear_read_error(stream=None) -> int:
    """Reads and clears the 4-bit linear's device error word, one for all streams (synchronises `stream`)."""
    code = ctypes.c_int32(0)
    _check(lib().moe_q4_linear_read_error(ctypes.byref(code), _stream(stream)), "moe_q4_linear_read_error")
    return code.value
