"""The example layer with an 8-bit cache and with a window, its two parts each against 64 bits (tests/layer_ref.py)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from layer_ref import Half, bound, cache_bound, heads_of  # noqa: E402
from q8_ref import from_codes, power  # noqa: E402
from test_gpu_decoder_layer import SIZES  # noqa: E402
from test_gpu_q8_layer import example  # noqa: E402, F401


def _held(layer, seq, n):
    """The k and v that the cache holds of a sequence's first n places, [n][kv heads][dim], 64 bits."""
    pages = layer.table[seq, :-(-n // layer.page_size)].long()
    values = [t.cpu() for t in layer.cache.tensors]
    if layer.scale_block:
        values = [from_codes(c.view(torch.uint8)) * power(s.int() - 127).repeat_interleave(layer.scale_block, 2)[..., None]
                  for c, s in zip(values[:2], values[2:])]
    return [c[pages].double().permute(0, 2, 1, 3).reshape(-1, layer.kv_heads, layer.dim)[:n] for c in values]


@pytest.mark.parametrize("block,window,sinks", [(16, None, 0), (8, 11, 2), (16, 40, 0), (16, 5, 1), (1, None, 0), (None, 11, 2), (None, 1, 0)])
@pytest.mark.parametrize("pieces", [[50], [20, 30], [33, 16, 1], [1] * 30])
def test_parts_agree_with_64_bits(example, pieces, block, window, sinks):  # noqa: F811
    layer = example.DecoderLayer(**SIZES, seed=4, scale_block=block, window=window, sinks=sinks)
    h = Half.of(layer)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    n = sum(pieces)
    x, other = (torch.randn(n, layer.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    at = 0
    for c in pieces:  # the sequence and another one in every step
        p = layer.plan({2: c, 0: c})
        layer.step(p, torch.cat([x[at:at + c], other[at:at + c]]))
        assert layer.errors(p) == (0, 0)
        for seq, rows, hs in ((2, x, p["hs"][:c]), (0, other, p["hs"][c:])):
            rows = rows[:at + c].cpu()
            held = _held(layer, seq, at + c)
            for got, want in zip(held, heads_of(h, rows, 0, False)[1:]):
                assert (got - want).norm() <= cache_bound(block is not None) * want.norm()
            if c > 1 or at > 10:  # a row alone has few elements, the first ones few keys
                want, tol = bound(h, rows[at:], *held, at, window, sinks, block is not None)
                err = (hs.cpu().double() - rows[at:].double() - want).norm()
                assert err <= tol, (err, tol, want.norm())
        at += c
