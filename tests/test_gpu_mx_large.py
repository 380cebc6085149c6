"""The MXFP4 grouped GEMM's 256 x 256 tile in each of its forms (FP32 and BF16 results, gathered
rows, SwiGLU, the re-quantised result with and without C, weight gradients), and the layer at a
size where its products take that tile.  Every test states which tile the dispatch rule picks."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from oracle import mxfp4 as M
from tests.gpu_util import bf16_rne_of, dev_bf16, dev_f32, dev_i32, host, rel_frob, same_bits
from tests.test_gpu_mx import ULP, check_codes, check_product, vals

pytestmark = pytest.mark.gpu


def tile(rows, cols, E, group_k=False):
    """Rows of the tile that a product takes.  rows: of A (GROUP_K: the gradient's), cols: rows of B
    per expert (with SwiGLU gate and up)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    up = lambda n: (n + 255) // 256
    if group_k:
        return 256 if E * up(rows) * up(cols) >= cus else 128
    if rows >= 144 * E and (rows // 256 + E // 2) * up(cols) >= cus:
        return 256
    return 128 if rows >= 64 * E else 64


# an expert without rows, with one, with parts of a wave's 64 and of the tile's 256 rows, and with many tiles
COUNTS = [0, 1, 63, 9000, 0, 65, 255, 257, 300, 12500, 0]
E, OFF = len(COUNTS), np.concatenate([[0], np.cumsum(COUNTS)])
R = int(OFF[-1])


def operands(gpu_lib, K, n, gathered):
    """A (or 5000 tokens and their row indices), B, and the values that the product's rows take."""
    T = 5000
    x = synth.activations(T if gathered else R, K, K)
    idx = synth.rng(K).integers(0, T, R).astype(np.int32) if gathered else None
    aq = gpu_lib.mxfp4_quantize(dev_bf16(x))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * n, K), n)))
    av = vals(aq)
    return aq, bq, None if idx is None else dev_i32(idx), av if idx is None else av[idx]


# one, two, three and four stages of K = 256, the last one partly filled
@pytest.mark.parametrize("K", [32, 288, 672, 1024])
@pytest.mark.parametrize("epi,N", [(0, 700), (0, 641), (1, 352), (1, 321)])
@pytest.mark.parametrize("gathered", [False, True])
def test_products(gpu_lib, K, epi, N, gathered):
    n = N * (1 + epi)
    assert tile(R, n, E) == 256
    aq, bq, ri, av = operands(gpu_lib, K, n, gathered)
    o = dict(M_cap=R, a_rows=ri, epilogue=epi)
    C = torch.full((R + 3, N), 12345.0, dtype=torch.float32, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(OFF), E, N, C=C, **o)
    check_product(host(C)[:R], av, vals(bq), OFF, E, N, swiglu=bool(epi))
    assert (C[R:] == 12345.0).all()
    # BF16 is the FP32 result rounded to nearest even, in rows of any stride, and nothing else is written
    buf = torch.full((R, N + 6), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(OFF), E, N, C=buf[:, 1:1 + N], **o)
    assert np.array_equal(host(buf[:, 1:1 + N]), bf16_rne_of(host(C)[:R]))
    assert (buf[:, :1] == 9).all() and (buf[:, 1 + N:] == 9).all()
    # M_cap cuts the last rows off
    cut = torch.full((R, N), 7.0, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(OFF), E, N, C=cut, **{**o, "M_cap": R - 130})
    assert same_bits(cut[:R - 130], C[:R - 130]) and (cut[R - 130:] == 7).all()


@pytest.mark.parametrize("K", [32, 288, 672])
@pytest.mark.parametrize("N", [352, 384])   # with and without padding behind a row's scales
@pytest.mark.parametrize("rule", [M.FLOOR, M.CEIL])
@pytest.mark.parametrize("gathered", [False, True])
def test_requantised_swiglu(gpu_lib, K, N, rule, gathered):
    assert tile(R, 2 * N, E) == 256
    aq, bq, ri, av = operands(gpu_lib, K, 2 * N, gathered)
    o = dict(M_cap=R, a_rows=ri, epilogue=gpu_lib.NV4_EPI_SWIGLU, rule=rule)
    off = dev_i32(OFF)
    plain = gpu_lib.mxfp4_grouped_gemm(aq, bq, off, E, N, **o)
    check_product(host(plain), av, vals(bq), OFF, E, N, swiglu=True)
    alone = gpu_lib.MXFP4.empty(R, N)
    alone.scales.fill_(0xEE)
    assert gpu_lib.mxfp4_grouped_gemm(aq, bq, off, E, N, q_out=alone, want_c=False, **o) is None
    check_codes(alone, host(plain), rule)
    for dt in (torch.float32, torch.bfloat16):
        q = gpu_lib.MXFP4.empty(R, N)
        C = torch.full((R, N + 3), 9.0, dtype=dt, device="cuda")
        gpu_lib.mxfp4_grouped_gemm(aq, bq, off, E, N, C=C[:, :N], q_out=q, **o)
        assert same_bits(C[:, :N].contiguous(), plain.to(dt)) and (C[:, N:] == 9).all()
        assert same_bits(q.codes, alone.codes) and same_bits(q.scales, alone.scales)
    # rows behind M_cap are left as they were
    more = gpu_lib.MXFP4(torch.full((R, N // 2), 0xAA, dtype=torch.uint8, device="cuda"),
                         torch.full((R, alone.scales.shape[1]), 0xAA, dtype=torch.uint8, device="cuda"), R, N)
    cut = gpu_lib.MXFP4(more.codes[:R - 130], more.scales[:R - 130], R - 130, N)
    gpu_lib.mxfp4_grouped_gemm(aq, bq, off, E, N, q_out=cut, want_c=False, **{**o, "M_cap": R - 130})
    assert same_bits(cut.codes, alone.codes[:R - 130]) and same_bits(cut.scales, alone.scales[:R - 130])
    assert (more.codes[R - 130:] == 0xAA).all() and (more.scales[R - 130:] == 0xAA).all()


@pytest.mark.parametrize("N,Mc,experts", [(513, 300, 43), (256, 512, 128), (96, 1000, 70)])
def test_weight_gradients(gpu_lib, N, Mc, experts):
    """Empty ranges, ranges of one to eleven K = 128 parts, and one of eighty."""
    assert tile(N, Mc, experts, group_k=True) == 256
    r = synth.rng(N)
    counts = r.integers(0, 1400, experts)
    counts[r.random(experts) < 0.3] = 0
    counts[r.random(experts) < 0.1] = 1
    counts[[0, -1]], counts[experts // 2] = 0, 10200
    off = np.concatenate([[0], np.cumsum(counts)])
    rows = int(off[-1])
    g = torch.Generator("cuda").manual_seed(N)
    po = gpu_lib.mx_padded_offsets(dev_i32(off))

    def cols(n):  # n columns (quantised in whole blocks of 32, the surplus ones cut off)
        t = torch.randn(rows, (n + 31) // 32 * 32, device="cuda", generator=g).bfloat16()
        q = gpu_lib.mxfp4_quantize(t, layout=gpu_lib.NV4_COLS, nseg=experts, seg_offsets=dev_i32(off),
                                   seg_padded_offsets=po)
        return gpu_lib.MXFP4(q.codes[:n], q.scales[:n], n, q.K)

    aq, bq = cols(N), cols(Mc)
    rpo = M.padded_offsets(off)
    P = int(rpo[-1])
    aq.scales[:, P // 32:] = 255   # NaN bytes behind the last segment must not matter
    C = gpu_lib.mxfp4_grouped_gemm(aq, bq, po, experts, 0, group_mode=gpu_lib.NV4_GROUP_K)
    av, bv = vals(aq)[:, :P], vals(bq)[:, :P]
    got = host(C)
    for e in range(experts):
        lo, hi = int(rpo[e]), int(rpo[e + 1])
        ref = av[:, lo:hi] @ bv[:, lo:hi].T
        tol = np.abs(av[:, lo:hi]) @ np.abs(bv[:, lo:hi]).T * (ULP * max(hi - lo, 1))
        assert (np.abs(got[e] - ref) <= tol).all(), e   # (an empty range: zeros)
    C16 = gpu_lib.mxfp4_grouped_gemm(aq, bq, po, experts, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=torch.bfloat16)
    assert np.array_equal(host(C16), bf16_rne_of(got))
    assert same_bits(C, gpu_lib.mxfp4_grouped_gemm(aq, bq, po, experts, 0, group_mode=gpu_lib.NV4_GROUP_K))


def test_layer_forward_and_backward(gpu_lib):
    """A prompt: every stage on the GPU's own inputs, most experts with some hundred rows, one with
    many and one with none."""
    T, H, n, k, I = 4096, 1024, 32, 4, 480
    R = T * k
    assert tile(R, 2 * I, n) == tile(R, H, n) == 256
    assert tile(H, I, n, group_k=True) == tile(2 * I, H, n, group_k=True) == 256
    r = synth.rng(7)
    X = synth.activations(T, H, 1)
    lg = synth.logits_softmax(T, n, 2)
    lg[:, 3] += 2.0
    lg[:, 9] -= 50.0
    W13, W2 = synth.weights((n, 2 * I, H), 3), synth.weights((n, H, I), 4)
    dY2, dY13 = synth.gradients((R, H), 5), synth.gradients((R, 2 * I), 6)
    w = gpu_lib.mx_quantize_expert_weights(dev_bf16(W13), dev_bf16(W2))
    wt = gpu_lib.mx_quantize_expert_weights_t(dev_bf16(W13), dev_bf16(W2))
    ids, wts = moe.route_topk(lg, k)
    p = moe.permute(ids, n)
    off, rt = p["offsets"], p["row_token"]
    assert np.diff(off).min() == 0 and np.diff(off).max() > 1000
    f = gpu_lib.mx_alloc_forward(T, H, n, k, I, keep_hact=True, out_dtype=torch.float32)
    gpu_lib.mx_moe_forward(dev_bf16(X), dev_f32(lg), w, k, f)
    check_codes(f.xq, X)
    assert np.array_equal(host(f.routing.row_token), rt)
    h32 = gpu_lib.mxfp4_grouped_gemm(f.xq, w.w13, f.routing.offsets, n, I, M_cap=R, a_rows=f.routing.row_token,
                                     epilogue=gpu_lib.NV4_EPI_SWIGLU)
    check_product(host(h32), vals(f.xq)[rt], vals(w.w13), off, n, I, swiglu=True)
    check_codes(f.hq, host(h32))
    assert np.array_equal(host(f.hact), bf16_rne_of(host(h32)))
    check_product(host(f.y), vals(f.hq), vals(w.w2), off, n, H)
    assert rel_frob(host(f.out), moe.combine(host(f.y), p["token_row"], wts)) <= 1e-5
    # without the kept SwiGLU output: the same rows
    assert same_bits(gpu_lib.mx_moe_forward(dev_bf16(X), dev_f32(lg), w, k).y, f.y)
    g = gpu_lib.mx_alloc_backward(T, H, n, k, I, dgrad_dtype=torch.float32)
    gpu_lib.mx_moe_backward(dev_bf16(X), f, wt, dev_bf16(dY2), dev_bf16(dY13), g)
    check_codes(g.dy2q, dY2)
    check_codes(g.dy13q, dY13)
    check_product(host(g.dhact), vals(g.dy2q), vals(wt.w2t), off, n, I)
    check_product(host(g.dxperm), vals(g.dy13q), vals(wt.w13t), off, n, H)
    po = M.padded_offsets(off)
    P = int(po[-1])
    col = lambda q: vals(q)[:, :P]
    for q, t in ((g.dy2c, dY2), (g.hc, host(f.hact)), (g.dy13c, dY13), (g.xc, X[rt])):
        assert np.array_equal(col(q), M.rounded(M.by_segment(np.asarray(t, np.float64), off)))
    for got, a, b in ((g.dw2, g.dy2c, g.hc), (g.dw13, g.dy13c, g.xc)):
        ref = moe.grouped_gemm_k(col(a), col(b), po, n)
        tol = moe.grouped_gemm_k(np.abs(col(a)), np.abs(col(b)), po, n) * ULP * (np.diff(po).max())
        assert (np.abs(host(got) - ref) <= tol).all()
    g16 = gpu_lib.mx_moe_backward(dev_bf16(X), f, wt, dev_bf16(dY2), dev_bf16(dY13))
    assert np.array_equal(host(g16.dhact), bf16_rne_of(host(g.dhact)))
    assert np.array_equal(host(g16.dxperm), bf16_rne_of(host(g.dxperm)))
    assert same_bits(g16.dw2, g.dw2) and same_bits(g16.dw13, g.dw13)
