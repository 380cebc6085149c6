"""The router's losses and gradients and the combine's gradients on the GPU against the FP64 oracle."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from oracle import router as R
from tests.gpu_util import dev_bf16, dev_f32, dev_i32, host, same_bits

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24


def case(T, E, k, nseg, pad, seed):
    r = synth.rng(seed)
    l = (r.standard_normal((T, E)) * 1.5 + r.standard_normal(E)).astype(np.float32)
    ids, _ = moe.route_topk(l, k) if T else (np.zeros((0, k), np.int32), None)
    mask = r.random(T) >= pad if pad else None
    off = np.concatenate([[0], np.sort(r.integers(0, T + 1, nseg - 1)), [T]]) if nseg else None
    return l, np.asarray(ids, np.int32), mask, off, r


def dev_mask(mask):
    return None if mask is None else torch.from_numpy(mask).cuda()


# A probability exp(l - max) / sum: the exponent's rounding and exp's own error (|l - max| <= 2^5 here: 32
# half steps and 2), the sum's E roundings, the quotient's: relative.
def p_tol(E):
    return (32 + 4 + E) * HALF


def check(lib, l, ids, mask, off, dloss, dw, renorm):
    T, E = l.shape
    k = ids.shape[1]
    so = None if off is None else dev_i32(off)
    lg, idd, m = dev_f32(l), dev_i32(ids), dev_mask(mask)
    b = lib.moe_balance_loss(lg, idd, mask=m, seg_offsets=so)
    ref = R.balance(l, ids, mask, off)
    assert np.array_equal(host(b.counts), ref["counts"]) and np.array_equal(host(b.tokens), ref["tokens"])
    # sums of T positive terms in FP32: at most T roundings in a chain
    rel = p_tol(E) + T * HALF
    assert (np.abs(host(b.prob_sums) - ref["prob_sums"]) <= rel * ref["prob_sums"] + 1e-37).all()
    # lse: off by the relative error of the sum, by log's and by its own rounding, squared and summed
    rel_z = 2 * (p_tol(E) + 4 * HALF * (1 + np.abs(R.softmax(l)[1]).max(initial=0))) + (T + 8) * HALF
    zabs = np.array([rel + (E + 12) * HALF, 0]) * np.abs(ref["loss"]) + np.array([0, rel_z * (2 + ref["loss"][1])])
    assert (np.abs(host(b.loss) - ref["loss"]) <= zabs + 1e-37).all()
    again = lib.moe_balance_loss(lg, idd, mask=m, seg_offsets=so)
    assert all(same_bits(x, y) for x, y in zip(vars(b).values(), vars(again).values()))
    g = lib.moe_balance_backward(lg, idd, b, None if dloss is None else dev_f32(dloss),
                                 dtopk_w=None if dw is None else dev_f32(dw), mask=m, seg_offsets=so,
                                 flags=lib.NV4_RENORM if renorm else 0)
    d = R.balance_backward(l, ids, ref["counts"], ref["tokens"], dloss, dw, renorm, mask, off)
    # every term is a product of a few factors, each within p_tol, E terms summed: against the sum of the
    # terms' magnitudes
    p, lse = R.softmax(l) if T else (np.zeros((0, E)), np.zeros(0))
    mag = np.zeros((T, E))
    if dloss is not None and T:
        seg = np.zeros(T, int) if off is None else np.searchsorted(off[1:], np.arange(T), side="right")
        n = len(ref["tokens"])
        seg = np.minimum(seg, n - 1)        # (a token behind the last segment has no such terms)
        n_t = np.maximum(ref["tokens"], 1)[seg][:, None]
        c = ref["counts"][seg].astype(np.float64)
        mag += abs(dloss[0]) * E / (n * k * n_t ** 2.0) * p * (c + (c * p).sum(1, keepdims=True))
        mag += abs(dloss[1]) * 2 / (n * n_t) * np.abs(lse)[:, None] * p
    if dw is not None and T:
        w = np.take_along_axis(p, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        a = np.abs(w * dw)
        q = np.zeros((T, E))
        for j in range(k):
            q[np.arange(T), ids[:, j]] += a[:, j] + w[:, j] * a.sum(1)
        mag += q if renorm else q + p * a.sum(1, keepdims=True)
    tol = (3 * p_tol(E) + (E + 16) * HALF) * mag
    assert (np.abs(host(g) - d) <= tol + 1e-37).all(), float(np.max(np.abs(host(g) - d) / (tol + 1e-37)))
    return b, g


@pytest.mark.parametrize("T,E,k,nseg,pad", [(1, 1, 1, 0, 0), (1, 8, 2, 1, 0), (2, 3, 3, 5, 0.5), (31, 32, 4, 2, 0), (33, 33, 1, 3, .3),
                                            (257, 60, 4, 3, 0.2), (65, 64, 6, 0, 0), (300, 128, 8, 7, 0.1),
                                            (129, 129, 32, 1, 0), (70, 256, 8, 40, 0.9), (50, 300, 7, 2, 0),
                                            (40, 512, 8, 1, 0.5), (20, 1000, 5, 3, 0), (9, 1024, 8, 1, 0), (3000, 17, 2, 90, 0.2)])
@pytest.mark.parametrize("renorm", [False, True])
def test_losses_and_gradients(gpu_lib, T, E, k, nseg, pad, renorm):
    l, ids, mask, off, r = case(T, E, k, nseg, pad, T + E)
    dw = r.standard_normal((T, k)).astype(np.float32)
    check(gpu_lib, l, ids, mask, off, np.array([0.7, 0.3], np.float32), dw, renorm)


@pytest.mark.parametrize("dloss,weights", [(None, True), (True, False), (None, False)])
def test_either_gradient_alone(gpu_lib, dloss, weights):
    l, ids, mask, off, r = case(200, 40, 4, 3, 0.3, 5)
    dw = r.standard_normal(ids.shape).astype(np.float32) if weights else None
    _, g = check(gpu_lib, l, ids, mask, off, np.array([1.0, -2.0], np.float32) if dloss else None, dw, False)
    if not dloss and not weights:
        assert (g == 0).all()


def test_gradient_against_differences(gpu_lib):
    """The GPU's own losses, differenced in a few directions: the z loss is smooth on the scale of a step
    of 2^-6 and FP32 losses resolve it."""
    l, ids, mask, off, r = case(64, 16, 2, 2, 0.2, 3)
    so, m, idd = dev_i32(off), dev_mask(mask), dev_i32(ids)
    for which in (0, 1):
        dl = np.eye(2, dtype=np.float32)[which]
        b = gpu_lib.moe_balance_loss(dev_f32(l), idd, mask=m, seg_offsets=so)
        g = host(gpu_lib.moe_balance_backward(dev_f32(l), idd, b, dev_f32(dl), mask=m, seg_offsets=so)).astype(np.float64)
        for s in range(3):
            v = synth.rng(s).standard_normal(l.shape).astype(np.float32)
            h = 2.0 ** -6
            f = [float(gpu_lib.moe_balance_loss(dev_f32(l + x * v), idd, mask=m, seg_offsets=so).loss[which]) for x in (h, -h)]
            num = (f[0] - f[1]) / (2 * h)
            # the third derivative along v: under 8 |v|_inf^3 times the loss; FP32 losses: 2^-20 of them over h
            size = max(f[0], 1.0)
            assert abs(num - (g * v).sum()) <= size * (h * h / 6 * 8 * np.abs(v).max() ** 3 + 2.0 ** -20 / h)


def test_infinite_logits_and_masked_nan(gpu_lib):
    """Experts switched off by -infinity or the lowest value, a token without any, NaN in a masked token."""
    l, ids, mask, off, r = case(90, 20, 3, 2, 0.3, 9)
    l[:, 5] = -np.inf
    l[:, 6] = np.finfo(np.float32).min
    ids, _ = moe.route_topk(np.where(np.isneginf(l), np.float32(-3e38), l), 3)
    ids = ids.astype(np.int32)
    live, dead = np.flatnonzero(mask)[3], np.flatnonzero(~mask)[1]
    l[live] = -np.inf
    l[dead] = np.nan
    dw = r.standard_normal(ids.shape).astype(np.float32)
    dw[dead] = 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    so = dev_i32(off)
    for renorm in (0, 1):
        b = gpu_lib.moe_balance_loss(dev_f32(l), dev_i32(ids), mask=dev_mask(mask), seg_offsets=so, dev_status=st)
        g = gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), b, dev_f32(np.ones(2)), dtopk_w=dev_f32(dw),
                                         mask=dev_mask(mask), seg_offsets=so, flags=renorm, dev_status=st)
        clean = np.where(np.isnan(l), 0, l)
        ref = R.balance(clean, ids, mask, off)
        assert st.item() == 0
        assert np.allclose(host(b.loss), ref["loss"], rtol=1e-5) and np.array_equal(host(b.counts), ref["counts"])
        d = R.balance_backward(clean, ids, ref["counts"], ref["tokens"], np.ones(2), dw, bool(renorm), mask, off)
        assert np.isfinite(host(g)).all() and (host(g)[[live, dead]] == 0).all() and (host(g)[:, 5] == 0).all()
        assert np.abs(host(g) - d).max() <= 1e-5
    # without the mask the NaN shows: in its segment's sums, its own gradient and the status
    b = gpu_lib.moe_balance_loss(dev_f32(l), dev_i32(ids), seg_offsets=so, dev_status=st)
    assert st.item() == gpu_lib.NV4_DS_NAN_LOGIT and torch.isnan(b.loss).all()
    st.zero_()
    l[dead] = np.inf
    gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), b, dev_f32(np.ones(2)), seg_offsets=so, dev_status=st)
    assert st.item() == gpu_lib.NV4_DS_NAN_LOGIT


def test_bad_ids_and_the_same_twice(gpu_lib):
    l, ids, mask, off, r = case(50, 12, 3, 2, 0, 4)
    ids[3, 1] = ids[3, 0]
    dw = r.standard_normal(ids.shape).astype(np.float32)
    check(gpu_lib, l, ids, mask, off, np.array([1, 1], np.float32), dw, True)
    check(gpu_lib, l, ids, mask, off, np.array([1, 1], np.float32), dw, False)
    ids[7, 2], ids[8, 0] = -1, 12
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    so = dev_i32(off)
    b = gpu_lib.moe_balance_loss(dev_f32(l), dev_i32(ids), seg_offsets=so, dev_status=st[:1])
    ref = R.balance(l, ids, mask, off)
    assert np.array_equal(host(b.counts), ref["counts"]) and np.allclose(host(b.loss), ref["loss"], rtol=1e-5)
    for renorm in (0, 1):
        g = gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), b, dev_f32(np.ones(2)), dtopk_w=dev_f32(dw),
                                         seg_offsets=so, flags=renorm, dev_status=st[1:])
        d = R.balance_backward(l, ids, ref["counts"], ref["tokens"], np.ones(2), dw, bool(renorm), mask, off)
        assert np.abs(host(g) - d).max() <= 1e-5
    assert st.tolist() == [gpu_lib.NV4_DS_BAD_EXPERT] * 2


def test_no_tokens_and_segments_that_leave_some_out(gpu_lib):
    z = lambda *s: torch.empty(*s, device="cuda")
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    for off in (None, dev_i32(np.zeros(4))):
        b = gpu_lib.moe_balance_loss(z(0, 8), ids, seg_offsets=off)
        assert all((v == 0).all() for v in vars(b).values())
        assert gpu_lib.moe_balance_backward(z(0, 8), ids, b, z(2), seg_offsets=off).shape == (0, 8)
    l, ids, _, _, r = case(100, 8, 2, 0, 0, 1)
    off = np.array([10, 40, 40, 77])
    check(gpu_lib, l, ids, None, off, np.array([1, 1], np.float32), r.standard_normal(ids.shape).astype(np.float32), False)
    check(gpu_lib, l, ids, np.zeros(100, bool), off, np.array([1, 1], np.float32), None, False)
    # borders outside the tokens, or not in order, stay within memory
    for off in ([-5, 40, 1000], [50, 20, 90], [100, 0, 0]):
        b = gpu_lib.moe_balance_loss(dev_f32(l), dev_i32(ids), seg_offsets=dev_i32(np.array(off)))
        gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), b, dev_f32(np.ones(2)), seg_offsets=dev_i32(np.array(off)))
    torch.cuda.synchronize()


def test_ranks_add_their_sums(gpu_lib):
    """Counts and tokens of two halves added give the gradient of the whole."""
    l, ids, _, _, _ = case(128, 16, 2, 0, 0, 8)
    one = gpu_lib.moe_balance_loss(dev_f32(l), dev_i32(ids))
    halves = [gpu_lib.moe_balance_loss(dev_f32(l[i:i + 64]), dev_i32(ids[i:i + 64])) for i in (0, 64)]
    both = gpu_lib.MoeBalance(None, *(getattr(halves[0], f) + getattr(halves[1], f) for f in ("counts", "prob_sums", "tokens")))
    assert torch.equal(both.counts, one.counts) and torch.equal(both.tokens, one.tokens)
    dl = dev_f32(np.ones(2))
    whole = gpu_lib.moe_balance_backward(dev_f32(l), dev_i32(ids), one, dl)
    part = gpu_lib.moe_balance_backward(dev_f32(l[64:]), dev_i32(ids[64:]), both, dl)
    assert same_bits(whole[64:].contiguous(), part)


def test_gradient_in_place(gpu_lib):
    l, ids, mask, off, r = case(200, 100, 4, 3, 0.3, 2)
    so, m = dev_i32(off), dev_mask(mask)
    lg = dev_f32(l)
    b = gpu_lib.moe_balance_loss(lg, dev_i32(ids), mask=m, seg_offsets=so)
    ref = gpu_lib.moe_balance_backward(lg, dev_i32(ids), b, dev_f32(np.ones(2)), mask=m, seg_offsets=so)
    gpu_lib.moe_balance_backward(lg, dev_i32(ids), b, dev_f32(np.ones(2)), mask=m, seg_offsets=so, out=lg)
    assert same_bits(lg, ref)


# ----------------------------------------------------------------------------- combine

@pytest.mark.parametrize("T,k,H", [(1, 1, 4), (3, 2, 100), (17, 8, 2048), (5, 9, 260), (4, 32, 1028), (33, 3, 4096), (2, 5, 8188)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
def test_combine_backward(gpu_lib, T, k, H, dt, yt):
    r = synth.rng(H)
    dout = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(dt).cuda()
    Y = torch.from_numpy(r.standard_normal((T * k + 2, H + 8)).astype(np.float32)).to(yt).cuda()[:, 4:H + 4]
    row = (r.permutation(T * k) + 1).reshape(T, k).astype(np.int32)      # row 0 and the last are nobody's
    w = r.random((T, k), dtype=np.float32)
    dY = torch.full((T * k + 2, H + 4), 5.0, dtype=yt, device="cuda")[:, :H]
    _, dw = gpu_lib.moe_combine_backward(dout, Y, dev_i32(row), dev_f32(w), dY=dY)
    ry, rw = R.combine_backward(host(dout), host(Y), row, w)
    got = host(dY).astype(np.float64)
    assert (got[[0, -1]] == 5).all()
    half = 2.0 ** -24 + (2.0 ** -8 if yt == torch.bfloat16 else 0)
    assert (np.abs(got - ry)[1:-1] <= half * np.abs(ry)[1:-1]).all()
    mag = R.combine_backward(np.abs(host(dout)), np.abs(host(Y)), row, w)[1]
    assert (np.abs(host(dw) - rw) <= H * HALF * mag).all()
    y2, none = gpu_lib.moe_combine_backward(dout, Y, dev_i32(row), dev_f32(w), want_dw=False)
    assert none is None and same_bits(y2[1:-1].contiguous(), dY[1:-1].contiguous())
    none, w2 = gpu_lib.moe_combine_backward(dout, Y, dev_i32(row), dev_f32(w), want_dy=False)
    assert none is None and same_bits(w2, dw)


def test_combine_backward_rows_outside(gpu_lib):
    T, k, H = 6, 2, 64
    r = synth.rng(1)
    dout, Y = dev_f32(r.standard_normal((T, H))), dev_f32(r.standard_normal((8, H)))
    row = np.array([[0, 1], [2, -1], [3, 8], [4, 2 ** 31 - 1], [5, -2 ** 31], [6, 7]], np.int32)
    w = r.random((T, k), dtype=np.float32)
    dY, dw = gpu_lib.moe_combine_backward(dout, Y, dev_i32(row), dev_f32(w))
    ry, rw = R.combine_backward(host(dout), host(Y), row, w)
    assert np.allclose(host(dY), ry, rtol=1e-6) and np.allclose(host(dw), rw, rtol=1e-4, atol=1e-5)
    assert (host(dw)[1:5, 1] == 0).all()


def test_combine_backward_is_moe_combines(gpu_lib):
    """Against the forward's own differences: linear in Y and in w, so a difference is the derivative."""
    T, k, H = 9, 3, 128
    r = synth.rng(2)
    Y, w, dout = (r.standard_normal(s).astype(np.float32) for s in ((T * k, H), (T, k), (T, H)))
    row = r.permutation(T * k).reshape(T, k).astype(np.int32)
    dY, dw = gpu_lib.moe_combine_backward(dev_f32(dout), dev_f32(Y), dev_i32(row), dev_f32(w))
    f = lambda y, ww: float((host(gpu_lib.moe_combine(dev_f32(y), dev_i32(row), dev_f32(ww), out_dtype=torch.float32))
                             .astype(np.float64) * dout).sum())
    for s in range(3):
        vy, vw = synth.rng(s).standard_normal(Y.shape), synth.rng(s + 9).standard_normal(w.shape)
        base = np.abs(host(dY) * vy).sum() + np.abs(host(dw) * vw).sum()
        assert abs(f(vy.astype(np.float32), w) - (host(dY) * vy).sum()) <= base * 2.0 ** -20
        assert abs(f(Y, vw.astype(np.float32)) - (host(dw) * vw).sum()) <= (base + np.abs(Y).sum() * 4) * 2.0 ** -20


@pytest.mark.parametrize("T,k,H", [(3, 2, 8), (17, 8, 2048), (5, 9, 264), (33, 3, 4096), (2, 12, 8184)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_combine_backward_of_aligned_bf16_rows(gpu_lib, T, k, H, dt):
    """Rows that allow 16-byte accesses give the bits that rows between such steps give."""
    r = synth.rng(H)
    dout = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(dt).cuda()
    Y = torch.from_numpy(r.standard_normal((T * k, H)).astype(np.float32)).bfloat16().cuda()
    row, w = dev_i32(r.permutation(T * k).reshape(T, k)), dev_f32(r.random((T, k), dtype=np.float32))
    dY, dw = gpu_lib.moe_combine_backward(dout, Y, row, w)
    ry, rw = R.combine_backward(host(dout), host(Y), host(row), host(w))
    assert (np.abs(host(dY) - ry) <= (2.0 ** -24 + 2.0 ** -8) * np.abs(ry)).all()
    mag = R.combine_backward(np.abs(host(dout)), np.abs(host(Y)), host(row), host(w))[1]
    assert (np.abs(host(dw) - rw) <= H * HALF * mag).all()
    between = torch.zeros(T * k, H + 4, dtype=torch.bfloat16, device="cuda")[:, 4:]
    between.copy_(Y)
    y2, w2 = gpu_lib.moe_combine_backward(dout, between, row, w)
    assert same_bits(y2.contiguous(), dY) and (np.abs(host(w2) - rw) <= H * HALF * mag).all()


# ----------------------------------------------------------------------------- many tokens

def many(T, E, k, seed):
    """Logits a good deal apart, choices by size (the first of a few tokens twice), a mask, and segments whose
    borders lie inside a wave's tokens, some of them empty."""
    r = synth.rng(seed)
    l = (3 * r.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(-l, 1, kind="stable")[:, :k].astype(np.int32)
    if k > 1:
        ids[5::97, 1] = ids[5::97, 0]
    mask = r.random(T) < 0.9
    off = np.sort(np.concatenate([[0, 3, 3, 5, T - 2], r.integers(0, T, 20), [T]])).astype(np.int32)
    return l, ids, mask, off, r


@pytest.mark.parametrize("T,E,k", [(16384, 7, 2), (16391, 60, 4), (20001, 128, 8), (16400, 130, 8), (16385, 260, 3), (16389, 600, 8)])
@pytest.mark.parametrize("renorm", [False, True])
def test_many_tokens(gpu_lib, T, E, k, renorm):
    l, ids, mask, off, r = many(T, E, k, T + E)
    dw = r.standard_normal((T, k)).astype(np.float32)
    dw[::3] = 0
    check(gpu_lib, l, ids, mask, off, np.array([0.7, 0.3], np.float32), dw, renorm)


@pytest.mark.parametrize("T", [40, 16390])
def test_arrays_between_16_byte_steps(gpu_lib, T):
    """The same bits where the arrays' starts do not allow wide accesses."""
    E, k = 128, 4
    l, ids, mask, off, r = many(T, E, k, 9)
    so, m, idd, dl = dev_i32(off), dev_mask(mask), dev_i32(ids), dev_f32(np.array([0.5, 2], np.float32))
    dw = dev_f32(r.standard_normal((T, k)).astype(np.float32))
    lg = dev_f32(l)
    odd = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    odd.copy_(lg)
    a, b = [gpu_lib.moe_balance_loss(x, idd, mask=m, seg_offsets=so) for x in (lg, odd)]
    assert all(same_bits(x, y) for x, y in zip(vars(a).values(), vars(b).values()))
    run = lambda x, **o: gpu_lib.moe_balance_backward(x, idd, a, dl, dtopk_w=dw, mask=m, seg_offsets=so, **o)
    g = run(lg)
    assert same_bits(run(odd, out=torch.empty(T * E + 1, device="cuda")[1:].view(T, E)), g)
    assert same_bits(run(odd, out=odd), g)
    a.counts = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), a.counts.flatten()])[1:].view_as(a.counts)
    assert same_bits(run(lg), g)


def test_many_empty_segments(gpu_lib):
    """65536 segments, most of them empty, for a few tokens and for many."""
    for T in (100, 16500):
        r = synth.rng(T)
        E, k, n = 8, 2, 65536
        l = r.standard_normal((T, E)).astype(np.float32)
        ids = np.argsort(-l, 1)[:, :k].astype(np.int32)
        off = np.sort(np.concatenate([[0], r.integers(0, T, n - 1), [T]])).astype(np.int32)
        check(gpu_lib, l, ids, None, off, np.array([500.0, 300.0], np.float32), None, False)
