"""The bounds of the tests of 8-bit attention, on the CPU: rounding probabilities to fp16 stays within them, rounding them to
bf16 does not."""
import pytest

torch = pytest.importorskip("torch")

from attn_ref import make_batch  # noqa: E402
from q8_bounds import attention8  # noqa: E402
from q8_ref import store  # noqa: E402

# (heads, kv_heads, dim, chunks, caches) of few keys: outputs far smaller than the values that they are made of, next to which
# their own rounding to bf16 does not count, are common there
FEW_KEYS = {
    "decode": (8, 2, 128, [1] * 24, [2 + i % 9 for i in range(24)]),
    "decode many rows": (32, 2, 64, [1] * 12, [2 + i % 9 for i in range(12)]),
    "chunks": (8, 1, 128, [40, 33, 20], [40, 35, 22]),
    "chunks dim 64": (16, 2, 64, [40, 33], [40, 35]),
}


def few_keys(name, seed=0):
    heads, kv_heads, dim, ql, kl = FEW_KEYS[name]
    return make_batch("bf16", heads, kv_heads, dim, 16, ql, kl, seed=seed)


@pytest.mark.parametrize("name", list(FEW_KEYS))
def test_the_bound_tells_fp16_probabilities_from_bf16(name):
    bt = few_keys(name)
    bt.k_cache, bt.v_cache = store(bt.k_cache, 16)[2], store(bt.v_cache, 16)[2]
    scale = bt.dim ** -0.5
    out, tol = attention8(bt, scale)
    rounded = lambda t: attention8(bt, scale, probabilities=t)[0].bfloat16().double()  # noqa: E731
    assert ((rounded(torch.float16) - out).abs() <= tol).all()
    over = (rounded(torch.bfloat16) - out).abs() > tol
    assert over.double().mean() > 1e-3, over.double().mean()
