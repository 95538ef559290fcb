"""Attention over the 8-bit cache on the GPU within the bounds of its own arithmetic (tests/q8_bounds.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from q8_bounds import attention8  # noqa: E402
from test_gpu_q8_cache import BATCH, Dev, _built  # noqa: E402, F401
from test_q8_bounds import FEW_KEYS, few_keys  # noqa: E402
from attn_ref import make_batch  # noqa: E402


def hold(bt, block, window=None, sinks=0, scale=None):
    """The kernel's outputs against the bound; the run's Dev."""
    d = Dev(bt, block)
    scale = bt.dim ** -0.5 if scale is None else scale
    d.attend(scale, window, sinks)
    assert d.errors() == 0
    out, tol = attention8(bt, scale, window, sinks)
    over = (d.out.cpu().double() - out).abs() - tol
    assert (over <= 0).all(), f"over the bound by {over.max()}, at {int((over > 0).sum())} of {over.numel()} elements"
    return d


@pytest.mark.parametrize("name", list(FEW_KEYS))
@pytest.mark.parametrize("block", [16, 1])
def test_few_keys(name, block):
    for seed in range(3):
        hold(few_keys(name, seed), block)
        hold(few_keys(name, seed), block, window=5, sinks=1)


@pytest.mark.parametrize("name", list(BATCH))
def test_all_sizes(name):
    spec = BATCH[name]
    hold(make_batch(*spec, seed=31), math.gcd(16, spec[4]))
    hold(make_batch(*spec, seed=32), spec[4], window=100, sinks=4)


def groups_apart(name, d, seed=0):
    """A batch whose groups of 16 keys lie 2^d apart, two and two of those in a step of every eight or so, and in which
    the small ones count all the same: the large ones' k and v fill the first half of a head only, of which the odd
    query heads see nothing."""
    bt = make_batch(*BATCH[name], seed=seed)
    g, half = torch.Generator().manual_seed(seed + 1), bt.dim // 2
    for c in (bt.k_cache, bt.v_cache):
        x = c.double().unflatten(2, (-1, 16))
        small = torch.rand(x.shape[:3], generator=g) < 0.5
        small[: x.shape[0] // 4] = False  # and steps with one kind only
        x[..., half:] = torch.where(small[..., None, None], x[..., half:], torch.zeros(()))
        x *= torch.where(small, 2.0 ** -d, 1.0)[..., None, None]
        c.copy_(x.flatten(2, 3))
    q = bt.q.double()
    q[:, ::2, half:], q[:, 1::2, :half] = 0, 0
    q[:, 1::2] *= 2.0 ** d
    bt.q.copy_(q)
    return bt


@pytest.mark.parametrize("name", ["decode ragged", "decode group 16", "few tokens", "chunk over cache", "chunk dim 64", "chunk ragged", "chunk fp32"])
def test_scales_apart(name):
    # on and beside the distances at which tiles take other units: 2^8, 2^15, 2^22 below the largest scale
    for d in (0, 1, 6, 7, 8, 9, 14, 15, 16, 17, 21, 22, 23, 24, 30):
        bt = groups_apart(name, d, seed=d)
        if torch.isnan(bt.q).any():
            pytest.fail("the case is wrong")
        hold(bt, 16)
        if d % 5 == 1:
            hold(bt, 16, window=150, sinks=20)


FAR = {
    # heads, kv_heads, dim, chunk, keys, window (None: all keys, of which no token's scores choose the large ones)
    "decode window": (4, 2, 128, 4, 400, 351),
    "decode window, many rows": (16, 4, 64, 4, 400, 351),
    "decode": (8, 2, 128, 1, 900, None),
    "decode, many rows": (24, 2, 64, 1, 900, None),
    "chunk window": (8, 1, 128, 200, 700, 455),
    "chunk window dim 64": (16, 2, 64, 200, 700, 455),
    "chunk": (8, 1, 128, 60, 700, None),
    "chunk dim 64": (16, 2, 64, 60, 700, None),
}


@pytest.mark.parametrize("name", list(FAR))
@pytest.mark.parametrize("power", [20, 36, 58, 75, 100])
def test_values_that_lie_far_apart(name, power):
    # keys 32 to 47 hold values 2^power larger than the others, those on to 255 nothing: with a window the first two
    # tokens see two and one of them, without one nobody gives them weight
    heads, kv_heads, dim, n, m, window = FAR[name]
    bt = make_batch("bf16", heads, kv_heads, dim, 16, [n], [m], seed=power)
    place = lambda p: (bt.table[0, p // 16].long(), slice(None), p % 16)  # noqa: E731
    g = torch.Generator().manual_seed(1)
    if window is None:
        bt.q[:] = torch.randn(dim, generator=g).bfloat16()
    for p in range(32, 256):
        bt.v_cache[place(p)] *= 2.0 ** power if p < 48 else 0.0
        if window is None and p < 48:
            bt.k_cache[place(p)] = -16 * bt.q[0, 0].sign()  # scores of about -16 * 0.8 * sqrt(dim)
    d = Dev(bt, 16)
    d.attend(dim ** -0.5, window, 0)
    assert d.errors() == 0
    got = d.out.cpu().double()
    assert got.isfinite().all()
    out, tol = attention8(bt, dim ** -0.5, window)
    seers = 2 if window else 0
    assert ((got - out).abs() <= tol)[:seers].all()
    if power < 60:  # the others as if the large values were not there
        largest = 2 * max(float(bt.v_cache[place(p)].abs().max()) for p in range(32, 48))
        for p in range(32, 48):
            bt.v_cache[place(p)] = 0.0
        out, tol = attention8(bt, dim ** -0.5, window)
        # but for keys 0 to 31, which lie within 128 keys of the large ones: a tile of a chunk holds their values times 2^-15 in fp16
        # and takes the rest into their probabilities, times 2^7, of which fp16 keeps what is above 2^-25: 2^-54 of the largest
        # value.  In decode a pair of steps has one unit, and probabilities times 2^14 and a scale's distance to it lose what
        # is below 2^-25: 2^-39.  A key's part is then off by that or, where it is smaller, by all of itself.
        least = 2.0 ** (-54 if n * heads // kv_heads > 16 else -39) * largest
        for p in range(m):
            bt.v_cache[place(p)] = bt.v_cache[place(p)].abs().clamp(max=least) if p < 32 else 0.0
        tol += attention8(bt, dim ** -0.5, window)[0]
        over = ((got - out).abs() - tol)[seers:]
        assert (over <= 0).all(), over.max()


BEFORE = {
    # heads, kv_heads, dim, chunk, keys: the last block of 16 keys holds large values, which only its own tokens see
    "decode": (4, 2, 128, 4, 401),
    "decode, many rows": (16, 4, 64, 4, 401),
    "decode long": (4, 2, 128, 4, 6001),
    "decode long, many rows": (16, 4, 64, 4, 6001),
    "chunk": (8, 1, 128, 60, 700),
    "chunk dim 64": (16, 2, 64, 60, 700),
    "chunk cut": (8, 1, 128, 60, 3000),
}


@pytest.mark.parametrize("name", list(BEFORE))
@pytest.mark.parametrize("power", [60, 90, 126, 127, 128, 135, 180])
def test_small_values_before_large_ones(name, power):
    # values of 2^-90 and, 2^power larger, those of the last block
    heads, kv_heads, dim, n, m = BEFORE[name]
    bt = make_batch("bf16", heads, kv_heads, dim, 16, [n], [m], seed=power)
    start = (m - 1) // 16 * 16
    place = lambda p: (bt.table[0, p // 16].long(), slice(None), p % 16)  # noqa: E731
    for p in range(m):
        bt.v_cache[place(p)] *= 2.0 ** (-90 if p < start else power - 90)
    d = Dev(bt, 16)
    d.attend(dim ** -0.5)
    assert d.errors() == 0
    got = d.out.cpu().double()
    seers = n - (m - start)  # the first row that sees the large values
    out, tol = attention8(bt, dim ** -0.5)
    assert ((got - out).abs() <= tol)[seers:].all()
    # the rows before: right, but for the keys that lie within 128 of the large ones, which may count as 0 (and, once they are
    # less than 2^-100 of them, all of them: fp32 then holds no part of them in units of the large ones)
    for p in range(start, m):
        bt.v_cache[place(p)] = 0.0
    out, tol = attention8(bt, dim ** -0.5)
    for p in range(m):
        bt.v_cache[place(p)] = bt.v_cache[place(p)].abs() if start - 128 <= p < start or power > 100 else 0.0
    tol += attention8(bt, dim ** -0.5)[0]
    over = ((got - out).abs() - tol)[:seers]
    assert (over <= 0).all(), over.max()
