"""Pins of the oracle's MXFP4: every E2M1 border under every scale, exact rational
arithmetic for the scale rules, and the layer's identity with a dense MLP."""

from fractions import Fraction

import numpy as np
import pytest

import synth
from oracle import formats as F
from oracle import moe
from oracle import mxfp4 as M


def _exponent(amax: Fraction, rule: int) -> int:
    """The rule by search over exact rationals."""
    if amax == 0:
        return -127
    e = -400
    if rule == M.FLOOR:
        while Fraction(2) ** (e + 1) <= amax:
            e += 1
        e -= 2
    else:
        while amax > 6 * Fraction(2) ** e:
            e += 1
    return max(e, -127)


@pytest.mark.parametrize("rule", [M.FLOOR, M.CEIL])
def test_scale_rule_against_rationals(rule):
    r = synth.rng(1)
    bits = r.integers(0, 0x7F800000, 4000).astype(np.uint32)
    edge = [0, 1, 2, 3, 0x007FFFFF, 0x00800000, 0x00C00000, 0x00C00001, 0x01000000, 0x01400000, 0x01400001, 0x7F7FFFFF,
            0x3F800000, 0x3FC00000, 0x3FC00001, 0x40C00000]
    a = np.concatenate([bits, np.array(edge, np.uint32)]).view(np.float32)
    got = M.scale_bytes(a.astype(np.float64), rule)
    for v, b in zip(a, got):
        assert int(b) == _exponent(Fraction(float(v)), rule) + 127


def test_borders_under_every_scale():
    """Each border, its FP32 neighbours and the saturation range, under each power of two that
    FP32 reaches, in a block whose maximum 4 * 2^e fixes the scale."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5], np.float32)
    want_tie = [0, 2, 2, 4, 4, 6]
    for e in range(-127, 125):
        s = np.ldexp(1.0, e)
        v = np.zeros(32)
        v[0] = 4 * s
        v[1:7] = borders * s
        if e > -100:
            v[7:13] = np.nextafter(borders, np.float32(10)) * s
            v[13:19] = -np.nextafter(borders, np.float32(0)) * s
        c, b = M.quantize(v[None])
        assert b[0, 0] == e + 127
        assert c[0, 0] == 6 and list(c[0, 1:7]) == want_tie
        if e > -100:
            assert list(c[0, 7:13]) == [1, 2, 3, 4, 5, 6] and list(c[0, 13:19]) == [8, 9, 10, 11, 12, 13]
    v = np.zeros((1, 32))
    v[0, :3] = [7.9, 6.5, -5.01]
    c, b = M.quantize(v)
    assert b[0, 0] == 127 and list(c[0, :3]) == [7, 7, 15]           # floor: saturates
    c, b = M.quantize(v, M.CEIL)
    assert b[0, 0] == 128 and list(c[0, :3]) == [6, 5, 13]           # 3.95, 3.25, -2.505 of 2


def test_special_blocks():
    v = np.zeros((4, 32))
    v[1, 5], v[2, 7] = np.inf, np.nan
    v[3] = -0.0
    c, b = M.quantize(v)
    assert list(b[:, 0]) == [0, 255, 255, 0] and (c[:3] == 0).all() and (c[3] == 8).all()
    assert np.isnan(M.values(c, b)[1:3]).all() and (M.values(c, b)[[0, 3]] == 0).all()


def test_values_are_nearest():
    """Brute force: no E2M1 value under the block's scale is nearer, saturation aside."""
    x = synth.activations(8, 256, 3)
    for rule in (M.FLOOR, M.CEIL):
        c, b = M.quantize(x, rule)
        grid = F.e2m1_decode(np.arange(16, dtype=np.uint8)).astype(np.float64)
        s = np.repeat(np.ldexp(1.0, b.astype(int) - 127), 32, 1)
        best = np.abs(grid[None, None] * s[..., None] - x[..., None]).min(-1)
        assert np.array_equal(np.abs(M.values(c, b) - x), best)


def test_by_segment_and_layer_identity():
    off = np.array([0, 3, 3, 131])
    x = synth.activations(131, 8, 5)
    t = M.by_segment(x, off)
    assert t.shape == (8, 256) and np.array_equal(M.padded_offsets(off), [0, 128, 128, 256])
    assert np.array_equal(t[:, :3], x[:3].T) and (t[:, 3:128] == 0).all() and np.array_equal(t[:, 128:], x[3:].T)
    # one expert, weight 1: a dense MLP on the rounded operands
    W13, W2 = synth.weights((1, 64, 64), 6), synth.weights((1, 64, 32), 7)
    xs = synth.activations(5, 64, 8)
    out, *_ = M.layer(xs, np.zeros((5, 1), int), np.ones((5, 1)), M.rounded(W13), M.rounded(W2))
    h = moe.swiglu(M.rounded(xs) @ M.rounded(W13)[0].T)
    assert np.allclose(out, M.rounded(h) @ M.rounded(W2)[0].T, rtol=1e-12, atol=0)
