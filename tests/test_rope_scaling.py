"""Frequencies of a scaled rotation at worked values: the blend between kept and divided pairs, its bounds,
and the gain."""
import math

import pytest


@pytest.fixture(scope="module")
def mx():
    from mxfp8_block_scaled_fa_gb300 import mxfa
    return mxfa


def share_kept(rp, base, factor):
    """Per pair x of f = plain (x + (1 - x) / factor)."""
    n = rp.turns.numel()
    ratio = [(int(t) % 2 ** 64) / 2 ** 64 * 2 * math.pi / base ** (-i / n) for i, t in enumerate(rp.turns)]
    return [(r - 1 / factor) / (1 - 1 / factor) for r in ratio]


# Pair i of n turns original / (2 pi) base^(-i / n) times, so `turns` times at i = n ln(original / (2 pi turns)) / ln(base):
#   n 64, base 1e4, original 4096:  32 times at 64 * 3.01436 / 9.21034 = 20.95, once at 64 * 6.48010 / 9.21034 = 45.03
#   n 32, base 1e6, original 32768: 32 times at 32 * 5.09380 / 13.81551 = 11.80, once at 32 * 8.55954 / 13.81551 = 19.83
@pytest.mark.parametrize("n,base,original,factor,low,high", [(64, 1e4, 4096, 32.0, 20, 46), (32, 1e6, 32768, 4.0, 11, 20)])
def test_yarn_blend_between_whole_pairs(mx, n, base, original, factor, low, high):
    rp = mx.Rope.make(2 * n, base, scaling="yarn", factor=factor, original=original, device="cpu")
    want = [min(1.0, max(0.0, (high - i) / (high - low))) for i in range(n)]
    # a frequency is off by half a 2^-64 of a turn at most: 2^-62 radians, below 1e-12 of the slowest here, 1e-6
    assert share_kept(rp, base, factor) == pytest.approx(want, abs=1e-9)
    assert rp.gain == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-12)


def test_yarn_values_by_hand(mx):
    rp = mx.Rope.make(128, scaling="yarn", factor=32.0, device="cpu")
    kept = share_kept(rp, 1e4, 32.0)
    assert kept[20] == pytest.approx(1.0) and kept[46] == pytest.approx(0.0, abs=1e-9)
    assert kept[36] == pytest.approx(10 / 26) and kept[45] == pytest.approx(1 / 26)


def test_yarn_choices(mx):
    make = lambda **kw: mx.Rope.make(128, scaling="yarn", factor=8.0, device="cpu", **kw)
    # bounds between pairs: linear in the logarithm of a pair's turns
    exact = share_kept(make(rounded=False), 1e4, 8.0)
    turns = [4096 / (2 * math.pi) * 1e4 ** (-i / 64) for i in range(64)]
    assert exact == pytest.approx([min(1.0, max(0.0, math.log(t) / math.log(32))) for t in turns], abs=1e-9)
    # other bounds: 64 and 2 turns at 64 * 2.32121 / 9.21034 = 16.13 and 64 * 5.78695 / 9.21034 = 40.21
    other = share_kept(make(fast=64.0, slow=2.0), 1e4, 8.0)
    assert other == pytest.approx([min(1.0, max(0.0, (41 - i) / 25)) for i in range(64)], abs=1e-9)
    assert make(gain=1.25).gain == 1.25 and mx.Rope.make(64, gain=0.5, device="cpu").gain == 0.5
    # every pair faster than `slow`, and none: bounds within the pairs' own range
    assert share_kept(mx.Rope.make(16, scaling="yarn", factor=4.0, original=1 << 30, device="cpu"), 1e4, 4.0)[0] == pytest.approx(1.0)
    few = share_kept(mx.Rope.make(16, scaling="yarn", factor=4.0, original=1, device="cpu"), 1e4, 4.0)
    assert few[1:] == pytest.approx([0.0] * 7, abs=1e-9)
    for bad in (dict(fast=1.0, slow=1.0), dict(fast=1.0, slow=2.0), dict(slow=0.0), dict(gain=float("nan")), dict(gain=float("inf"))):
        with pytest.raises(ValueError):
            make(**bad)
