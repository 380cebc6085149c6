"""Pins of the router oracle: hand-made cases, brute force, and differences of the losses."""

import numpy as np
import pytest

import synth
from oracle import moe
from oracle import router as R


def case(T=23, E=9, k=3, nseg=3, seed=1):
    r = synth.rng(seed)
    l = r.standard_normal((T, E))
    ids, _ = moe.route_topk(l.astype(np.float32), k)
    mask = r.random(T) < 0.7
    off = np.concatenate([[0], np.sort(r.integers(0, T + 1, nseg - 1)), [T]])
    return l, ids, mask, off, r


def test_even_routing_has_balance_one():
    """Every expert chosen equally often and uniform probabilities: 1; z is (ln E)^2."""
    E, k, T = 8, 2, 16
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    b = R.balance(np.zeros((T, E)), ids)
    assert (b["counts"] == T * k // E).all() and np.allclose(b["loss"], [1.0, np.log(E) ** 2], rtol=1e-15)
    # all on one expert with all the probability: E / k ... of one choice
    l = np.full((T, E), -np.inf)
    l[:, 3] = 2.0
    b = R.balance(l, np.full((T, 1), 3))
    assert np.allclose(b["loss"], [E, 4.0])


def test_sums_and_a_segment_without_tokens():
    l, ids, mask, off, _ = case()
    off = np.array([0, 5, 5, 23])
    b = R.balance(l, ids, mask, off)
    assert b["tokens"].sum() == mask.sum() and (b["counts"].sum(1) == 3 * b["tokens"]).all()
    assert np.allclose(b["prob_sums"].sum(1), b["tokens"])
    assert b["tokens"][1] == 0 and (b["counts"][1] == 0).all()
    two = R.balance(l, ids, mask, np.array([0, 5, 23]))
    assert np.allclose(b["loss"] * 3, two["loss"] * 2)


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    l, ids, mask, off, r = case()
    ids[2, 1] = ids[2, 0]                                      # the same expert twice
    dw, dloss = r.standard_normal(ids.shape), np.array([0.7, 0.3])
    b = R.balance(l, ids, mask, off)

    def total(l):
        v = (R.balance(l, ids, mask, off)["loss"] * dloss).sum()
        p, _ = R.softmax(l)
        w = np.take_along_axis(p, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return v + (w * dw).sum()

    g = R.balance_backward(l, ids, b["counts"], b["tokens"], dloss, dw, renorm, mask, off)
    h = 1e-5
    for t in range(len(l)):
        for e in range(l.shape[1]):
            d = np.zeros_like(l)
            d[t, e] = h
            # the third derivative of these sums is below 10: h^2 / 6 * 10, and 1e-15 / h of cancellation
            assert abs((total(l + d) - total(l - d)) / (2 * h) - g[t, e]) < 2e-9


def test_combine_gradients_are_the_adjoint():
    r = synth.rng(5)
    T, k, H = 7, 3, 12
    Y, w, dout = r.standard_normal((T * k, H)), r.standard_normal((T, k)), r.standard_normal((T, H))
    row = r.permutation(T * k).reshape(T, k)
    dY, dw = R.combine_backward(dout, Y, row, w)
    DY, Dw = r.standard_normal(Y.shape), r.standard_normal(w.shape)
    assert np.isclose((dout * moe.combine(DY, row, w)).sum(), (dY * DY).sum(), rtol=1e-12)
    assert np.isclose((dout * moe.combine(Y, row, Dw)).sum(), (dw * Dw).sum(), rtol=1e-12)


def test_tokens_without_probabilities():
    l, ids, mask, off, r = case()
    l[4] = -np.inf
    mask[4] = True
    b = R.balance(l, ids, mask, off)
    assert np.isfinite(b["loss"]).all()
    dw = r.standard_normal(ids.shape)
    for renorm in (False, True):
        g = R.balance_backward(l, ids, b["counts"], b["tokens"], np.ones(2), dw, renorm, mask, off)
        assert np.isfinite(g).all() and (g[4] == 0).all()
