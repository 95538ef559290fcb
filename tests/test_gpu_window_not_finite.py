"""Keys and values that are not finite, at a place that the first token of a chunk sees and the others' windows have left."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from attn_ref import make_batch  # noqa: E402
from q8_ref import attention  # noqa: E402
from test_gpu_q8_cache import BATCH, Dev, _built  # noqa: E402, F401

WINDOW = 30


@pytest.mark.parametrize("name", ["few tokens", "chunk over cache", "chunk dim 64", "chunk ragged", "chunk many long", "chunk fp32", "odd pages", "odd head size"])
@pytest.mark.parametrize("block", [None, 16, 8])
@pytest.mark.parametrize("what", ["k nan", "k inf", "v nan", "v inf"])
def test_who_they_reach(name, block, what):
    if block and "inf" in what:
        pytest.skip("codes have no infinity")
    bt = make_batch(*BATCH[name], seed=23)
    block = block and math.gcd(block, bt.page)
    b = max(range(len(bt.q_len)), key=lambda i: bt.q_len[i] if bt.kv_len[i] - bt.q_len[i] >= WINDOW - 1 else 0)
    n, m, t, group = bt.q_len[b], bt.kv_len[b], int(bt.cu_q[b]), bt.heads // bt.kv_heads
    assert n > 1
    p = m - n - WINDOW + 1  # the first key of the first token's window
    d = Dev(bt, block)
    out, lse, tol, tol_lse = attention(bt, 0.1, WINDOW, 0)
    cache = d.k if what[0] == "k" else d.v
    bad = (math.nan if "nan" in what else math.inf) if block is None else 0xff
    cache[int(bt.table[b, p // bt.page]), 0, p % bt.page, 5] = bad
    d.attend(0.1, WINDOW, 0)
    assert d.errors() == 0
    got, got_lse = d.out.cpu().double(), d.lse.cpu().double()
    first = torch.zeros(bt.tokens, bt.heads, dtype=torch.bool)
    first[t, :group] = True
    if what[0] == "k":
        if "nan" in what:
            assert got[first].isnan().all() and got_lse[first].isnan().all()
        others = ~first
    else:
        assert not got[first][:, 5].isfinite().any() and ((got_lse - lse).abs() <= tol_lse)[~lse.isinf()].all()
        others = torch.ones_like(first)
        others[t:t + n, :group] = False
        own = got[t:t + n, :group]  # of the same chunk: right, or not finite in that element
        good = (own - out[t:t + n, :group]).abs() <= tol[t:t + n, :group]
        good[..., 5] |= ~own[..., 5].isfinite()
        assert good.all()
    assert ((got - out).abs() <= tol)[others].all()
