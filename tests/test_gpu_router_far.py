"""The gradient of renormalised routing weights where the chosen experts' logits lie far below the row's largest:
a selection by biased or grouped scores chooses such experts, and their weights are a softmax of their own."""

import numpy as np
import pytest
import torch

import synth
from tests.gpu_util import dev_f32, dev_i32, host, same_bits

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24


def renormalised(l, ids, dw):
    """sum over the choices m of expert j of w_m (dw_m - sum_i w_i dw_i), in 64 bits, and the sum of the terms'
    magnitudes; choices whose logits are all -infinity have no weights."""
    v = np.take_along_axis(l.astype(np.float64), ids, 1)
    mx = v.max(1, keepdims=True)
    e = np.exp(v - np.where(np.isneginf(mx), 0.0, mx))
    z = e.sum(1, keepdims=True)
    w = e / np.where(z == 0, 1.0, z)
    a = w * dw
    d, mag = np.zeros(l.shape), np.zeros(l.shape)
    for j in range(ids.shape[1]):
        rows = np.arange(len(l))
        d[rows, ids[:, j]] += a[:, j] - w[:, j] * a.sum(1)
        mag[rows, ids[:, j]] += np.abs(a[:, j]) + w[:, j] * np.abs(a).sum(1)
    return d, mag


def case(T, E, k, gap, seed):
    """Random choices, lowered by `gap` below where they were drawn; every ninth token keeps its largest logits,
    every eleventh names an expert twice."""
    r = synth.rng(seed)
    l = r.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(r.random((T, E)), 1)[:, :k].astype(np.int32)
    low = l.copy()
    np.put_along_axis(low, ids, np.take_along_axis(l, ids, 1) - np.float32(gap), 1)
    ids[::9] = np.argsort(-l[::9], 1)[:, :k]
    low[::9] = l[::9]
    if k > 1:
        ids[4::11, 1] = ids[4::11, 0]
    return low, ids, r.standard_normal((T, k)).astype(np.float32)


# A weight is exp(l - max) / sum over k choices that differ by less than 2^4: the difference's rounding (16 half
# steps of the result), exp's own two steps, k sums, the quotient's reciprocal and product; then a few products
# and the sum over E experts' terms.
def tol(E, k):
    return 3 * (16 + 4 + k + 3) * HALF + (E + 16) * HALF


@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (37, 7, 3), (64, 64, 2), (130, 128, 8), (45, 200, 5), (33, 1024, 32), (16390, 64, 4)])
@pytest.mark.parametrize("gap", [0, 80, 86.9, 88, 104, 200, 3e4])
def test_choices_far_below_the_largest(gpu_lib, T, E, k, gap):
    l, ids, dw = case(T, E, k, gap, T + E)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda x, **o: gpu_lib.moe_balance_backward(x, dev_i32(ids), dtopk_w=dev_f32(dw), flags=gpu_lib.NV4_RENORM,
                                                      dev_status=st, **o)
    g = run(dev_f32(l))
    d, mag = renormalised(l, ids, dw)
    assert np.isfinite(host(g)).all()
    # (weights under FP32's smallest normal number may be 0)
    assert (np.abs(host(g) - d) <= tol(E, k) * mag + 2.0 ** -125 * np.abs(dw).sum(1, keepdims=True)).all()
    assert st.item() == 0
    x = dev_f32(l)
    assert same_bits(run(x, out=x), g)


def test_beside_the_losses_and_without_any_weight(gpu_lib):
    """The losses' part is what it is without the weights; choices of -infinity alone have no weights."""
    T, E, k = 50, 40, 3
    l, ids, dw = case(T, E, k, 120, 1)
    np.put_along_axis(l[7:8], ids[7:8], -np.inf, 1)
    l[8] = -np.inf
    lg, idd, dl = dev_f32(l), dev_i32(ids), dev_f32(np.array([0.5, 0.25]))
    b = gpu_lib.moe_balance_loss(lg, idd)
    both = host(gpu_lib.moe_balance_backward(lg, idd, b, dl, dtopk_w=dev_f32(dw), flags=gpu_lib.NV4_RENORM)).astype(np.float64)
    losses = host(gpu_lib.moe_balance_backward(lg, idd, b, dl)).astype(np.float64)
    d, mag = renormalised(l, ids, dw)
    assert np.isfinite(both).all()
    # each part within its own bound, and the sum's rounding
    assert (np.abs(both - losses - d) <= tol(E, k) * mag + 4 * HALF * (np.abs(losses) + np.abs(d)) + 1e-35).all()
    assert (both[8] == 0).all() and (both[7, ids[7]] == 0).all()


def test_chosen_nan_and_infinity(gpu_lib):
    """A NaN or infinity among the choices or beside them makes its token's row NaN, and no other's."""
    T, E, k = 40, 24, 3
    l, ids, dw = case(T, E, k, 100, 2)
    bad = {3: np.nan, 5: np.inf, 12: np.nan, 13: np.inf}
    for t, v in bad.items():
        out = [e for e in range(E) if e not in ids[t]]
        l[t, ids[t, 1] if t < 10 else out[0]] = v
    g = host(gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), dtopk_w=dev_f32(dw), flags=gpu_lib.NV4_RENORM))
    rows = sorted(bad)
    assert np.isnan(g[rows]).all() and np.isfinite(np.delete(g, rows, 0)).all()
