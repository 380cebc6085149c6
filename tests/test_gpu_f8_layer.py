"""The FP8 layer and the router's training side as they are used together: every stage of a training step on
the GPU's own inputs, streams, graphs, and sizes behind 32 bits."""

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as M
from oracle import moe
from oracle import mxfp4 as MX
from oracle import router as R
from tests.gpu_util import bf16_rne_of, dev_bf16, dev_f32, dev_i32, host, rel_frob, same_bits
from tests.test_gpu_f8 import CUT, HALF_BF16, ULP, check_codes, check_product, same_floats, tile_vals, vals
from tests.test_gpu_mx_streams import keep_busy, pool_of
from tests.test_gpu_router import check as check_balance

pytestmark = pytest.mark.gpu


def check_cols(q, x, off, rule):
    """Codes and scales of a segment-wise transpose; columns behind the last segment are not looked at."""
    xt = MX.by_segment(np.asarray(x, np.float64), off) if q.K else None
    P = int(MX.padded_offsets(off)[-1])
    c, G = M.quantize(xt[:, :P].astype(np.float32), rule)
    assert np.array_equal(host(q.codes)[:, :P], c) and same_floats(host(q.scales)[:, :P // 128], G)


def step(lib, x, lg, w, wt, k, dout, dloss, f, g, seq=None, flags=0, dY13=None):
    """A training step's calls: the forward, the losses, and the gradients back to the router's logits."""
    lib.fp8_moe_forward(x, lg, w, k, f, flags=flags)
    rt = f.routing
    b = lib.moe_balance_loss(lg, rt.topk_ids, seg_offsets=seq)
    dy, dw = lib.moe_combine_backward(dout, f.y, rt.token_row, rt.topk_w)
    lib.fp8_moe_backward(x, f, wt, dy, dY13, g)
    dlg = lib.moe_balance_backward(lg, rt.topk_ids, b, dloss, dtopk_w=dw, seg_offsets=seq, flags=flags)
    return [f.out, g.dhact, g.dxperm, g.dw2, g.dw13, b.loss, b.counts, dw, dlg]


@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
@pytest.mark.parametrize("T,E,k,H,I,renorm", [(96, 8, 2, 256, 128, False), (5, 16, 4, 160, 96, True),
                                             (700, 12, 3, 272, 224, True), (1, 4, 4, 128, 32, False)])
def test_training_step_stage_by_stage(gpu_lib, T, E, k, H, I, renorm, rule):
    r = synth.rng(T)
    X, lgh = synth.activations(T, H, 1), synth.logits_softmax(T, E, 2)
    W13, W2 = synth.weights((E, 2 * I, H), 3), synth.weights((E, H, I), 4)
    dout, dY13h = synth.gradients((T, H), 5), synth.gradients((T * k, 2 * I), 6)
    w = gpu_lib.fp8_quantize_expert_weights(dev_bf16(W13), dev_bf16(W2), rule=rule)
    wt = gpu_lib.fp8_transpose_expert_weights(w)
    flags = gpu_lib.NV4_RENORM if renorm else 0
    f = gpu_lib.fp8_alloc_forward(T, H, E, k, I, keep_hact=True, out_dtype=torch.float32, rule=rule)
    g = gpu_lib.fp8_alloc_backward(T, H, E, k, I, dgrad_dtype=torch.float32)
    x, lg, dloss = dev_bf16(X), dev_f32(lgh), np.array([0.01, 0.001], np.float32)
    out, dhact, dx, dw2, dw13, loss, counts, dtw, dlg = step(gpu_lib, x, lg, w, wt, k, dev_f32(dout), dev_f32(dloss), f, g,
                                                            flags=flags, dY13=dev_bf16(dY13h))
    ids, wts = moe.route_topk(lgh, k, renorm)
    p = moe.permute(ids, E)
    off, rows = p["offsets"], T * k
    rt = f.routing
    assert np.array_equal(host(rt.topk_ids), ids) and np.array_equal(host(rt.token_row), p["token_row"])
    # forward
    check_codes(f.xq, X, rule)
    gate = tile_vals(w.w13)
    h32 = gpu_lib.fp8_grouped_gemm(f.xq, w.w13, rt.offsets, E, I, M_cap=rows, a_rows=rt.row_token,
                                   epilogue=gpu_lib.NV4_EPI_SWIGLU)
    check_product(host(h32), vals(f.xq)[p["row_token"]], gate, off, E, I, swiglu=True)
    check_product(host(f.hact), vals(f.xq)[p["row_token"]], gate, off, E, I, swiglu=True, bf16=True)
    # (codes of the unrounded result: half a BF16 step and half a code step from hact)
    hv, hb = vals(f.hq), host(f.hact).astype(np.float64)
    G = np.repeat(host(f.hq.scales).astype(np.float64), 128, 1)[:, :I]
    assert (np.abs(hv - hb) <= HALF_BF16 * np.abs(hb) + (2.0 ** -4 * np.abs(hv) + 2.0 ** -10 * G) * (1 + 1e-6)).all()
    check_product(host(f.y), hv, tile_vals(w.w2), off, E, H)
    assert rel_frob(host(out), moe.combine(host(f.y), p["token_row"], wts)) <= 1e-5
    # losses, and the gradients of the combine and of the logits
    ref = R.balance(lgh, ids)
    assert np.array_equal(host(counts), ref["counts"]) and np.allclose(host(loss), ref["loss"], rtol=1e-5)
    ry, rw = R.combine_backward(dout, host(f.y), p["token_row"], host(rt.topk_w))
    mag = R.combine_backward(np.abs(dout), np.abs(host(f.y)), p["token_row"], host(rt.topk_w))[1]
    assert (np.abs(host(dtw) - rw) <= H * 2.0 ** -24 * mag).all()
    _, again = check_balance(gpu_lib, lgh, ids, None, None, dloss, host(dtw), renorm)
    assert same_bits(again, dlg)
    # the layer's backward
    dY2 = gpu_lib.moe_combine_backward(dev_f32(dout), f.y, rt.token_row, rt.topk_w, want_dw=False)[0]
    assert (np.abs(host(dY2) - ry) <= 2.0 ** -23 * np.abs(ry)).all()
    check_codes(g.dy2q, host(dY2), rule)
    check_codes(g.dy13q, dY13h, rule)
    w2t, w13t = tile_vals(wt.w2t), tile_vals(wt.w13t)
    assert same_floats(w2t.reshape(E, I, H), tile_vals(w.w2).reshape(E, H, I).transpose(0, 2, 1))
    check_product(host(dhact), vals(g.dy2q), w2t, off, E, I)
    check_product(host(dx), vals(g.dy13q), w13t, off, E, H)
    for q, t in ((g.dy2c, host(dY2)), (g.hc, host(f.hact)), (g.dy13c, dY13h), (g.xc, X[p["row_token"]])):
        check_cols(q, t, off, rule)
    po = MX.padded_offsets(off)
    P = int(po[-1])
    col = lambda q: M.values(host(q.codes)[:, :P], host(q.scales)[:, :P // 128])
    longest = int(np.diff(po).max())
    for got, a, b in ((dw2, g.dy2c, g.hc), (dw13, g.dy13c, g.xc)):
        ref = moe.grouped_gemm_k(col(a), col(b), po, E)
        tol = moe.grouped_gemm_k(np.abs(col(a)), np.abs(col(b)), po, E) * ULP * (longest + 3 * (longest // 128 + 1))
        assert (np.abs(host(got) - ref) <= tol).all()


def test_forward_without_buffers_and_refusals(gpu_lib):
    T, E, k, H, I = 20, 8, 2, 256, 64
    x, lg = dev_bf16(synth.activations(T, H, 1)), dev_f32(synth.logits_softmax(T, E, 2))
    w = gpu_lib.fp8_quantize_expert_weights(dev_bf16(synth.weights((E, 2 * I, H), 3)), dev_bf16(synth.weights((E, H, I), 4)))
    f = gpu_lib.fp8_moe_forward(x, lg, w, k)
    g = gpu_lib.fp8_alloc_forward(T, H, E, k, I, keep_hact=True)
    assert same_bits(gpu_lib.fp8_moe_forward(x, lg, w, k, g).out, f.out) and f.hact is None
    with pytest.raises(ValueError, match="keep_hact"):
        gpu_lib.fp8_moe_backward(x, f, gpu_lib.fp8_transpose_expert_weights(w), None, None)
    with pytest.raises(ValueError, match="bufs"):
        gpu_lib.fp8_moe_forward(x[:5], lg[:5], w, k, g)
    with pytest.raises(ValueError, match="columns"):
        gpu_lib.fp8_moe_forward(x[:, :128].contiguous(), lg, w, k)


def case(gpu_lib, T=96, E=8, k=2, H=256, I=64):
    lg = dev_f32(synth.logits_softmax(T, E, 2))
    x = dev_bf16(synth.activations(T, H, 1))
    g = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, dtype=torch.bfloat16, device="cuda", generator=g)
    w = gpu_lib.fp8_quantize_expert_weights(rand(E, 2 * I, H), rand(E, H, I))
    return x, lg, w, gpu_lib.fp8_transpose_expert_weights(w), rand(T, H), rand(T * k, 2 * I), (T, H, E, k, I)


def test_outputs_come_from_the_streams_pool(gpu_lib):
    x, lg, w, wt, dout, dY13, shape = case(gpu_lib)
    T, H, E, k, I = shape
    s = torch.cuda.Stream()
    rt = gpu_lib.moe_permute(lg, E, k)
    torch.cuda.synchronize()
    o = dict(stream=s)
    q = gpu_lib.fp8_quantize(x, **o)
    t = gpu_lib.fp8_transpose(w.w2, **o)
    b = gpu_lib.moe_balance_loss(lg, rt.topk_ids, **o)
    y = gpu_lib.fp8_grouped_gemm(q, w.w13, rt.offsets, E, 2 * I, M_cap=T * k, a_rows=rt.row_token, **o)
    outs = [q.codes, q.scales, gpu_lib.fp8_dequantize(q, **o), t.codes, t.scales, y, b.loss, b.counts, b.prob_sums, b.tokens,
            gpu_lib.moe_balance_backward(lg, rt.topk_ids, b, torch.ones(2, device="cuda"), **o),
            *gpu_lib.moe_combine_backward(dout, torch.ones(T * k, H, device="cuda"), rt.token_row, rt.topk_w, **o)]
    assert [pool_of(v) for v in outs] == [s.cuda_stream] * len(outs)
    f = gpu_lib.fp8_moe_forward(x, lg, w, k, **o)
    assert [pool_of(v) for v in (f.out, f.y, f.pws, f.xq.codes, f.hq.scales, f.routing.offsets)] == [s.cuda_stream] * 6
    torch.cuda.synchronize()


def test_calls_beside_a_busy_stream(gpu_lib):
    """The step on two streams in turn, each call's memory dropped while its kernels are pending."""
    x, lg, w, wt, dout, dY13, shape = case(gpu_lib)
    T, H, E, k, I = shape

    def one(s=None):
        with torch.cuda.stream(s):
            f = gpu_lib.fp8_alloc_forward(*shape, keep_hact=True)
            g = gpu_lib.fp8_alloc_backward(*shape)
            return step(gpu_lib, x, lg, w, wt, k, dout, torch.full((2,), 0.5, device="cuda"), f, g, dY13=dY13)

    want = one()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        keep_busy()
        got += [one(), one(s), one(s), one()]
    torch.cuda.synchronize()
    for ts in got:
        assert all(same_bits(a, b) for a, b in zip(ts, want))


def test_captured_and_replayed(gpu_lib):
    """The whole step in one graph, replayed with other inputs between eager steps: equal each time, also after
    batches that leave experts empty."""
    x, lg, w, wt, dout, dY13, shape = case(gpu_lib)
    T, H, E, k, I = shape
    seq = dev_i32(np.array([0, 40, 40, T]))
    dloss = torch.full((2,), 0.5, device="cuda")
    bufs = lambda: (gpu_lib.fp8_alloc_forward(*shape, keep_hact=True), gpu_lib.fp8_alloc_backward(*shape))
    eager, captured = bufs(), bufs()
    run = lambda fg: step(gpu_lib, x, lg, w, wt, k, dout, dloss, *fg, seq=seq, dY13=dY13)
    run(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(captured)
    for i in range(4):
        x.copy_(dev_bf16(synth.activations(T, H, 100 + i)))
        lg.copy_(dev_f32(synth.logits_softmax(T, E, 200 + i)))
        if i == 2:
            lg[:, 2:] -= 50      # every token to the same two experts
        want = [t.clone() for t in run(eager)]
        torch.cuda.synchronize()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, want))


def test_graphs_that_share_a_workspace(gpu_lib):
    """Two captured losses and an eager one in one workspace, in turn."""
    E, k = 60, 4
    lg = dev_f32(synth.logits_softmax(3000, E, 1))
    ids = gpu_lib.moe_permute(lg, E, k).topk_ids
    seq = {T: dev_i32(np.array([0, T // 3, T // 3, T])) for T in (1, 257, 3000)}
    ws = torch.empty(gpu_lib.load().moe_balance_workspace(3000, E, 3), dtype=torch.uint8, device="cuda")
    run = lambda T, **o: gpu_lib.moe_balance_loss(lg[:T], ids[:T], seg_offsets=seq[T], **o)
    want = {T: run(T) for T in seq}
    out, graphs = {T: run(T) for T in seq}, {}
    for T in seq:
        graphs[T] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[T]):
            run(T, ws=ws, out=out[T])
    for T in (3000, 1, 257, 3000, 257, 1, 1, 3000):
        for t in vars(out[T]).values():
            t.zero_()
        ws.fill_(0xFF)
        graphs[T].replay()
        got = run(257, ws=ws)
        torch.cuda.synchronize()
        for a, b in ((out[T], want[T]), (got, want[257])):
            assert all(same_bits(u, v) for u, v in zip(vars(a).values(), vars(b).values()))


# ----------------------------------------------------------------------------- sizes behind 32 bits

def test_rows_behind_32_bits(gpu_lib):
    """More than 2^32 bytes of every large operand but A's codes: the last rows against a call with those alone."""
    K, rows, tail = 2048, (1 << 20) + 4096 + 77, 300
    x = torch.randn(rows, K, device="cuda", dtype=torch.bfloat16)
    q, t = gpu_lib.fp8_quantize(x), gpu_lib.fp8_quantize(x[-tail:])
    assert x.numel() * 2 > 1 << 32 and same_bits(q.codes[-tail:], t.codes) and same_bits(q.scales[-tail:], t.scales)
    f32 = gpu_lib.fp8_dequantize(q, torch.float32)
    assert torch.equal(f32[-tail:], gpu_lib.fp8_dequantize(t, torch.float32))
    off, one = dev_i32(np.array([0, rows - tail, rows])), dev_i32(np.array([0, tail]))
    po = gpu_lib.mx_padded_offsets(off)
    seg = dict(nseg=2, seg_offsets=off, seg_padded_offsets=po)
    ref = gpu_lib.fp8_quantize(x[-tail:], layout=gpu_lib.NV4_COLS, nseg=1, seg_offsets=one,
                               seg_padded_offsets=gpu_lib.mx_padded_offsets(one))
    start, end = po[1].item(), po[2].item()
    c = gpu_lib.fp8_quantize(x, layout=gpu_lib.NV4_COLS, **seg)
    assert torch.equal(c.codes[:, start:end], ref.codes[:, :end - start])
    assert torch.equal(c.scales[:, start // 128:end // 128], ref.scales[:, :(end - start) // 128])
    del f32, c, x
    w = gpu_lib.fp8_quantize(torch.randn(2 * 2048, K, device="cuda", dtype=torch.bfloat16),
                             layout=gpu_lib.NV4_F8_TILES, nseg=2)
    q = gpu_lib.FP8(q.codes, q.scales, rows, K)
    second = gpu_lib.FP8(w.codes[2048:], w.scales[1:], 2048, K, 1)
    y = gpu_lib.fp8_grouped_gemm(q, w, off, 2, 2048)
    ref = gpu_lib.fp8_grouped_gemm(t, second, one, 1, 2048)
    assert y.numel() * 4 > 1 << 32
    # (another kernel may sum K in another order: K roundings against a sum of terms a hundred times a random row's)
    assert ((y[-tail:] - ref).norm(dim=1) <= K * 2.0 ** -24 * 100 * ref.norm(dim=1)).all()


def test_weights_above_4_gib(gpu_lib):
    """Experts on either side of 4 GiB of codes, by each kernel, against the same two experts alone."""
    E, N, K = 132, 8192, 4096
    codes = torch.randint(0, 127, (E * N, K), dtype=torch.uint8, device="cuda")
    scales = torch.rand(E, N // 128, K // 128, device="cuda")
    assert codes.numel() > 1 << 32
    w = gpu_lib.FP8(codes, scales, E * N, K, E)
    two = gpu_lib.FP8(torch.cat([codes[:N], codes[-N:]]), scales[[0, -1]].contiguous(), 2 * N, K, 2)
    for R in (2, 80, 700):
        x = gpu_lib.fp8_quantize(torch.randn(R, K, device="cuda", dtype=torch.bfloat16))
        far = dev_i32(np.array([0] + [R // 2] * (E - 1) + [R]))
        got = gpu_lib.fp8_grouped_gemm(x, w, far, E, N)
        ref = gpu_lib.fp8_grouped_gemm(x, two, dev_i32(np.array([0, R // 2, R])), 2, N)
        tol = K * 2.0 ** -24 * 100
        assert ((got - ref).norm(dim=1) <= tol * ref.norm(dim=1)).all() and ref.abs().max() > 0
    # the transpose of the last expert
    t = gpu_lib.fp8_transpose(w)
    assert torch.equal(t.codes[-K:], codes[-N:].T) and torch.equal(t.scales[-1], scales[-1].T)


def test_router_behind_32_bits(gpu_lib):
    """Logits and expert rows of more than 4 GiB: the last tokens against those alone."""
    E, k, T, tail = 128, 2, (1 << 23) + 4001, 1000
    lg = torch.randn(T, E, device="cuda")
    assert lg.numel() * 4 > 1 << 32
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    seq = dev_i32(np.array([0, T - tail, T]))
    b = gpu_lib.moe_balance_loss(lg, ids, seg_offsets=seq)
    one = gpu_lib.moe_balance_loss(lg[-tail:].contiguous(), ids[-tail:].contiguous())
    assert torch.equal(b.counts[1], one.counts[0]) and b.tokens.tolist() == [T - tail, tail]
    # (sums in another order: tail roundings)
    assert ((b.prob_sums[1] - one.prob_sums[0]).abs() <= tail * 2.0 ** -23 * one.prob_sums[0]).all()
    dl = torch.tensor([0.5, 0.25], device="cuda")
    g = gpu_lib.moe_balance_backward(lg, ids, b, dl, seg_offsets=seq)
    ref = gpu_lib.moe_balance_backward(lg[-tail:].contiguous(), ids[-tail:].contiguous(), one, dl / 2)
    assert same_bits(g[-tail:].contiguous(), ref)       # (halves: nseg is 2 there, and exact)
    del lg, g
    rows, H, T = (1 << 20) + 300, 2048, 400
    Y = torch.randn(rows, H, dtype=torch.bfloat16, device="cuda")
    assert Y.numel() * 2 > 1 << 32
    row = torch.stack([torch.arange(T), rows - 1 - torch.arange(T)], 1).int().cuda()
    dout, w = torch.randn(T, H, device="cuda"), torch.rand(T, 2, device="cuda")
    dY, dw = gpu_lib.moe_combine_backward(dout, Y, row, w)
    near = torch.cat([Y[:T], Y[-T:]])
    row2 = torch.stack([torch.arange(T), 2 * T - 1 - torch.arange(T)], 1).int().cuda()
    dY2, dw2 = gpu_lib.moe_combine_backward(dout, near, row2, w)
    assert same_bits(dw, dw2) and same_bits(torch.cat([dY[:T], dY[-T:]]), dY2)
