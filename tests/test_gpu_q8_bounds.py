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
