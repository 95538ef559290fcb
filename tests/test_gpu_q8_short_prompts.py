"""Many short prompts over an 8-bit cache: items of one step of keys that fill two tiles of query rows and one tile in turn, so
that a CTA's roles pass from item to item as often as they can."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from attn_ref import make_batch  # noqa: E402
from test_gpu_q8_cache import _built, check  # noqa: E402, F401


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("longest", [100, 900])
@pytest.mark.parametrize("chunks", [[45], [32, 16, 45, 3, 17], [16, 33]])
def test_items_of_two_tiles_and_of_one_in_turn(dim, longest, chunks):
    # groups of 8: a tile holds 16 tokens, an item 32.  Up to 512 keys a sequence no item is cut; one of 900 has items
    # cut where a CTA's share ends.
    n = 320
    ql = [chunks[i % len(chunks)] for i in range(n)]
    kl = [q + (i * 11) % (100 - q + 1) for i, q in enumerate(ql)]
    ql[n // 2], kl[n // 2] = 40, longest
    d = check(make_batch("bf16", 16, 2, dim, 16, ql, kl, seed=longest), block=16)
    first, first_lse = d.out.clone(), d.lse.clone()
    for _ in range(20):
        d.out.fill_(7.0)
        d.attend(dim ** -0.5)
    assert d.errors() == 0
    assert torch.equal(d.out, first) and torch.equal(d.lse, first_lse)


@pytest.mark.parametrize("dim", [64, 128])
def test_the_same_behind_windows(dim):
    ql = [[45, 20, 9][i % 3] for i in range(300)]
    kl = [q + (i * 29) % 400 for i, q in enumerate(ql)]
    check(make_batch("bf16", 16, 2, dim, 16, ql, kl, seed=dim), block=16, window=60, sinks=3)
