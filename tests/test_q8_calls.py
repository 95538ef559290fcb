"""What the binding of the 8-bit cache and the window refuses beside wrong sizes and types (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from test_q8_abi import FAKE, _on_gpu, _shape  # noqa: E402

POINTERS = {"16 bits": moe.MoEKVCache(FAKE, FAKE, 4096, 2048, 64),
            "8 bits": moe.MoEKVCacheQ8(FAKE, FAKE, FAKE, FAKE, 4096, 2048, 64, 4, 2, 16)}


def _call(name, cache, ws=None):
    """Call `name` with everything right but `cache` and the workspace (None: too small for any call)."""
    bf, i32 = torch.bfloat16, torch.int32
    q, k, v, out = (_on_gpu(torch.zeros(8, h, 64, dtype=bf)) for h in (8, 2, 2, 8))
    batch = moe.make_attn_batch(*(_on_gpu(torch.zeros(s, dtype=i32)) for s in (5, 4, (4, 5))))
    rope = moe.make_rope(64, device="cpu")
    rope.sizes = None
    if name == "append":
        moe.moe_rope_append(_shape(), rope, q, k, v, cache, batch, out, workspace=ws, stream=0)
    elif name == "append8":
        moe.moe_rope_append_q8(_shape(), rope, q, k, v, cache, batch, out, workspace=ws, stream=0)
    elif name == "attn":
        moe.moe_paged_attention(_shape(), q, cache, batch, out, workspace=ws, stream=0)
    elif name == "window":
        moe.moe_paged_attention_window(_shape(), q, cache, batch, moe.make_attn_window(5), out, workspace=ws, stream=0)
    else:
        moe.moe_paged_attention_q8(_shape(), q, cache, batch, out, workspace=ws, stream=0)


TAKES = {"append": "16 bits", "attn": "16 bits", "window": "16 bits", "append8": "8 bits", "attn8": "8 bits"}


@pytest.mark.parametrize("name", list(TAKES))
@pytest.mark.parametrize("kind", list(POINTERS))
def test_a_cache_put_together_by_hand_has_to_be_of_the_calls_kind(name, kind):
    if kind == TAKES[name]:
        with pytest.raises(moe.MoEError):  # the library's own refusal: no workspace
            _call(name, POINTERS[kind])
    else:
        with pytest.raises(ValueError, match="cache: a MoEKVCache"):
            _call(name, POINTERS[kind])


@pytest.mark.parametrize("name", list(TAKES))
def test_a_workspace_in_host_memory_is_refused(name):
    with pytest.raises(ValueError, match="workspace: not on the GPU"):
        _call(name, POINTERS[TAKES[name]], torch.zeros(1024, dtype=torch.uint8))  # too small: the library refuses it too
    with pytest.raises(moe.MoEError):
        _call(name, POINTERS[TAKES[name]], _on_gpu(torch.zeros(1024, dtype=torch.uint8)))


@pytest.mark.parametrize("value,kept", [(5, 5), (2**31 - 1, 2**31 - 1), (2**31, 2**31 - 1), (2**32 + 5, 2**31 - 1), (2**62, 2**31 - 1),
                                        (0, 0), (-1, -1), (-2**32 + 5, -1)])
def test_windows_past_32_bits_do_not_wrap(value, kept):
    w = moe.make_attn_window(value, value)
    assert (w.window, w.sinks) == (kept, kept)
