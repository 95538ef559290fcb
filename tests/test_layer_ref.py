"""The bounds of the layer tests, on the CPU: a layer that rounds where the example does is within them, one with a mistake
is not."""
import math

import pytest

torch = pytest.importorskip("torch")

from layer_ref import F16, Half, added, bound, cache_bound, heads_of  # noqa: E402
from q8_ref import store  # noqa: E402

SIZES = dict(hidden=256, heads=8, kv_heads=2, dim=64)


def _half(seed):
    """Weights as the example draws them, as dense ones."""
    g = torch.Generator().manual_seed(seed)
    hidden, wide = SIZES["hidden"], (SIZES["heads"] + 2 * SIZES["kv_heads"]) * SIZES["dim"]
    ones = lambda n: (1 + 0.1 * torch.randn(n, generator=g)).bfloat16()  # noqa: E731

    def dense(rows, cols):
        book = torch.tensor([-1 + 2 * j / 15 for j in range(16)], dtype=torch.float64)
        w = book[torch.randint(0, 16, (rows, cols), generator=g)]
        level = math.sqrt(float(book.square().mean()) * cols)
        return w * ((0.5 + torch.rand(rows, cols // 64, generator=g)) / level).double().repeat_interleave(64, 1)

    return Half(SIZES["heads"], SIZES["kv_heads"], SIZES["dim"], ones(hidden).double(), ones(64), ones(64), dense(wide, hidden),
                dense(hidden, SIZES["heads"] * SIZES["dim"]))


def _stored(x, block):
    """x [tokens][heads][dim] as an 8-bit cache holds it."""
    n = -(-len(x) // block) * block
    pages = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n - len(x))).transpose(0, 1)[None]  # [1][heads][slots][dim]
    return store(pages, block)[2][0].transpose(0, 1)[:len(x)]


@pytest.mark.parametrize("block,window,sinks", [(16, None, 0), (8, 11, 2), (16, 40, 0), (16, 5, 1), (1, None, 0)])
@pytest.mark.parametrize("n", [30, 50])
def test_mistakes_pass_the_bounds(block, window, sinks, n):
    h = _half(n)
    x = torch.randn(n, SIZES["hidden"], generator=torch.Generator().manual_seed(7)).bfloat16()
    _, k, v = heads_of(h, x, 0, False)
    near_q, near_k, near_v = heads_of(h, x, 0, True)
    kc, vc = _stored(near_k, block), _stored(near_v, block)
    # what the cache holds
    off = lambda got, want: float((got - want).norm() / want.norm())  # noqa: E731
    assert off(kc, k) < cache_bound(True) and off(vc, v) < cache_bound(True)
    unturned = heads_of(h, x, 0, True, turn=False)
    wrong = {"not rotated": (unturned[1], k), "shifted": (near_k.roll(1, 0), k), "the other head": (near_v.flip(1), v),
             "k for v": (near_k, v), "a scale doubled": (torch.cat([2 * vc[:16], vc[16:]]), v), "halved": (vc / 2, v)}
    for what, (got, want) in wrong.items():
        assert off(got, want) > cache_bound(True), what
    # what attention adds
    want, tol = bound(h, x, kc, vc, 0, window, sinks, True)
    near = lambda q=near_q, k=kc, v=vc, w=window, s=sinks, **kw: float((added(h, x, q, k, v, 0, w, s, F16, **kw) - want).norm())  # noqa: E731
    assert near() <= tol and tol < 0.05 * want.norm()
    wrong = {"nothing": float(want.norm()), "v halved": near(v=vc / 2), "v doubled": near(v=2 * vc), "q not rotated": near(q=unturned[0]),
             "k not rotated": near(k=_stored(unturned[1], block)), "k of zeros": near(k=0 * kc), "softmax's factor": near(scale=1.1),
             "the next key": near(later=1), "a scale doubled": near(v=torch.cat([2 * vc[:16], vc[16:]]))}
    if window is not None:
        wrong |= {"no window": near(w=None), "a window of one more": near(w=window + 1), "a first key more": near(s=sinks + 1)}
    for what, err in wrong.items():
        if (window, n, what) not in ((40, 30, "no window"), (40, 30, "a window of one more"), (40, 30, "a first key more")):
            assert err > tol, (what, err, tol)
