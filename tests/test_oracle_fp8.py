"""Pins of the FP8 oracle: exact rational arithmetic, torch's own E4M3 cast, and identities."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import synth
from oracle import formats as F
from oracle import fp8 as M


def test_codes_are_torchs_cast():
    """Every E4M3 midpoint and its FP32 neighbours, both signs, and a dense sweep."""
    v = F.e4m3_finite_nonneg().astype(np.float32)
    mid = ((v[1:].astype(np.float64) + v[:-1]) / 2).astype(np.float32)
    r = synth.rng(1)
    x = np.concatenate([v, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999)),
                        (r.random(20000) * np.exp2(r.integers(-14, 9, 20000))).astype(np.float32)])
    x = x[x <= 448]
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(M.encode(x), want)


def _exact_S(a: Fraction, rule: int) -> Fraction:
    if rule == M.POW2:
        t = 126
        while a * Fraction(2) ** t > 448:
            t -= 1
        return Fraction(2) ** t
    q, e = Fraction(448) / a, 0
    while q / Fraction(2) ** e >= 2:
        e += 1
    while q / Fraction(2) ** e < 1:
        e -= 1
    ulp = Fraction(2) ** (max(e, -126) - 23)
    n, rem = divmod(q, ulp)
    n += rem * 2 > ulp or (rem * 2 == ulp and n % 2 == 1)
    return min(n * ulp, Fraction(2) ** 126)


@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_factors_against_rationals(rule):
    r = synth.rng(2)
    bits = r.integers(1, 0x7F800000, 3000).astype(np.uint32)
    edge = [1, 2, 3, 0x007FFFFF, 0x00800000, 0x00E00000, 0x00E00001, 0x04E00000, 0x04E00001, 0x3F800000, 0x3FE00000,
            0x3FE00001, 0x43E00000, 0x43E00001, 0x7F7FFFFF]
    a = np.concatenate([bits, np.array(edge, np.uint32)]).view(np.float32)
    S, G = M.factors(a, rule)
    for v, s, g in zip(a, S, G):
        want = _exact_S(Fraction(float(v)), rule)
        assert Fraction(float(s)) == want
        # nothing saturates, and G is S's nearest reciprocal
        assert Fraction(float(v)) * want <= 448 * (1 + Fraction(2) ** -23)
        assert abs(Fraction(float(g)) * want - 1) <= Fraction(2) ** -24
    S, G = M.factors(np.array([0.0, np.inf, np.nan], np.float32), rule)
    assert S[0] == 1 and G[0] == 1 and np.isnan(G[1:]).all()


@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_error_bound_and_identities(rule):
    x = synth.to_bf16_values((synth.rng(3).standard_normal((9, 400)) * np.exp2(synth.rng(4).integers(-20, 20, (9, 1))))
                             .astype(np.float32))
    c, G = M.quantize(x, rule)
    v = M.values(c, G)
    top = np.repeat(np.maximum.reduceat(np.abs(x), [0, 128, 256, 384], axis=1), 128, 1)[:, :400]
    # half a step: 2^-4 of the value, and 2^-10 codes' worth below the normal codes (2^-9 / 2 of 1 / S)
    S = np.repeat(M.factors(np.maximum.reduceat(np.abs(x), [0, 128, 256, 384], axis=1), rule)[0], 128, 1)[:, :400]
    assert (np.abs(v - x) <= np.abs(x) * 2.0 ** -4 * (1 + 1e-6) + 2.0 ** -10 / S).all()
    assert (np.abs(v) <= top * (1 + 2.0 ** -3)).all()
    # blocks are independent, a power of two only moves the scales, and signs mirror
    c2, G2 = M.quantize(x[:, 128:], rule)
    assert np.array_equal(c2, c[:, 128:]) and np.array_equal(G2, G[:, 1:])
    c3, G3 = M.quantize(x * np.float32(2.0 ** 7), rule)
    assert np.array_equal(c3, c) and np.array_equal(G3, G * np.float32(2.0 ** 7))
    assert np.array_equal(M.quantize(-x, rule)[0], c ^ 0x80)


@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_tiles_are_row_blocks_of_one_scale_and_transpose(rule):
    x = synth.weights((300, 208), 5)
    c, G = M.quantize_tiles(x, rule)
    assert G.shape == (3, 2)
    ct, Gt = M.quantize_tiles(np.ascontiguousarray(x.T), rule)
    assert np.array_equal(ct, c.T) and np.array_equal(Gt, G.T)
    # a matrix whose every row holds the block's maximum quantises the same by rows
    y = x[:128, :128].copy()
    y[:, 0] = np.abs(y).max()
    cy, Gy = M.quantize_tiles(y, rule)
    cr, Gr = M.quantize(y, rule)
    assert np.array_equal(cy, cr) and (Gr == Gy[0, 0]).all()
    assert np.array_equal(M.tile_values(cy, Gy), M.values(cr, Gr))


def test_a_worked_example():
    """A = 7: S = 64; 3.5 -> 224, 1.3125 -> 84 (a tie between 80 and 88: the even code 80), -0 keeps its sign."""
    x = np.zeros((1, 16), np.float32)
    x[0, :5] = [7, 3.5, 1.3125, -0.0, 1.375]
    for rule in (M.FP32, M.POW2):
        c, G = M.quantize(x, rule)
        assert G[0, 0] == np.float32(1 / 64)
        assert list(F.e4m3_decode(c[0, :5])) == [448, 224, 80, 0, 88] and c[0, 3] == 0x80
    # A = 7.03125 (1.7578 * 4): the power of two halves
    x[0, 0] = 7.03125
    assert M.quantize(x, M.POW2)[1][0, 0] == np.float32(1 / 32)


def test_a_block_that_is_not_finite():
    x = np.ones((2, 256), np.float32)
    x[0, 3], x[1, 200] = np.nan, -np.inf
    c, G = M.quantize(x)
    assert np.isnan(G[0, 0]) and np.isnan(G[1, 1]) and G[0, 1] == G[1, 0] == np.float32(1) / np.float32(448)
    assert (c[0, :128] == 0).all() and (c[1, 128:] == 0).all()
    ct, Gt = M.quantize_tiles(x)
    assert np.isnan(Gt).all() and (ct == 0).all()
