"""GPU MXFP4 calls against the oracle: codes, scale bytes and permutations bit for bit; products
within the rounding of their FP32 sums; the few-token layer within that and the codes that such
a rounding can move; repeated, captured and side-stream calls bitwise equal."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from oracle import mxfp4 as M
from oracle import nvfp4 as Q
from tests.gpu_util import bf16_rne_of, dev_bf16, dev_f32, dev_i32, host, rel_frob, same_bits

pytestmark = pytest.mark.gpu

# An FP32 sum of n products is off by at most n - 1 roundings of partial sums, each at most
# 2^-24 of a partial sum of |products| when it rounds to nearest and 2^-23 when it truncates.
ULP = 2.0 ** -23
BF16_HALF = 2.0 ** -8  # half a BF16 step relative to the value


def unpacked(q):
    return Q.unpack_codes(host(q.codes)), host(q.scales)


def vals(q):
    return M.values(*unpacked(q))


def check_codes(q, x, rule=M.FLOOR):
    c, b = M.quantize(np.asarray(x, np.float64), rule)
    gc, gb = unpacked(q)
    nb = q.K // 32
    assert np.array_equal(gb[:, :nb], b), "scale bytes"
    assert (gb[:, nb:] == 0).all(), "scale padding"
    assert np.array_equal(gc, c), "codes"


def wide(shape, seed):
    """Values over the whole range of exponents a gradient meets, zeros and ties among them."""
    r = synth.rng(seed)
    x = r.standard_normal(shape) * np.exp2(r.integers(-30, 20, (shape[0], shape[1] // 32)).repeat(32, 1))
    x[r.random(shape) < 0.2] *= 0.0
    return synth.to_bf16_values(x.astype(np.float32))


# ----------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2048), (3, 96), (33, 160), (257, 1056), (1025, 2048), (4, 16416)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rule", [M.FLOOR, M.CEIL])
def test_quantize_rows(gpu_lib, rows, K, f32, rule):
    x = wide((rows, K), rows + K)
    if f32:
        x = x * (1 + synth.rng(9).random((rows, K), dtype=np.float32) * np.float32(1e-3))
    q = gpu_lib.mxfp4_quantize(dev_f32(x) if f32 else dev_bf16(x), rule=rule)
    check_codes(q, x, rule)
    for dt in (torch.bfloat16, torch.float32):
        assert np.array_equal(host(gpu_lib.mxfp4_dequantize(q, dt)).astype(np.float64), vals(q))


def test_quantize_extremes(gpu_lib):
    """Subnormal and largest blocks, negative zeros, NaN and infinity in a block."""
    x = np.zeros((8, 64), np.float32)
    x[0, :4] = [1e-45, -1e-45, 3e-45, 5e-44]
    x[1] = np.float32(9e-41)
    x[2, :3] = [3.4028235e38, -3.0e38, 1e38]
    x[3] = -0.0
    x[4, 3], x[5, 40], x[6, 2] = np.nan, np.inf, -np.inf
    x[4, 32:] = 1.0
    x[7, :5] = [1.1754944e-38, 2.3509887e-38, 4e-38, -6e-38, 1e-39]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (dev_f32(x), dev_bf16(x)):
        st.zero_()
        q = gpu_lib.mxfp4_quantize(t, dev_status=st)
        check_codes(q, t.float().cpu().numpy())
        assert st.item() == gpu_lib.NV4_DS_NONFINITE
        d = host(gpu_lib.mxfp4_dequantize(q))
        assert np.isnan(d[4, :32]).all() and np.isnan(d[5, 32:]).all() and np.isnan(d[6, :32]).all()
        assert np.isfinite(d[4, 32:]).all()
        st.zero_()
        gpu_lib.mxfp4_quantize(t[:4], dev_status=st)
        # (FP32's largest value is BF16's infinity)
        assert st.item() == (0 if t.dtype == torch.float32 else gpu_lib.NV4_DS_NONFINITE)


def test_quantize_strided_and_gathered(gpu_lib):
    x = wide((40, 192), 5)
    big = dev_bf16(np.concatenate([x, x[:, :64]], 1))
    check_codes(gpu_lib.mxfp4_quantize(big[:, 64:160]), x[:, 64:160])
    idx = np.array([39, 0, 7, 7, 21], np.int32)
    check_codes(gpu_lib.mxfp4_quantize(dev_bf16(x), row_index=dev_i32(idx)), x[idx])
    # an index outside x reads its nearest row
    q = gpu_lib.mxfp4_quantize(dev_bf16(x), row_index=dev_i32(np.array([-5, 99])))
    check_codes(q, x[[0, 39]])


SEGMENTS = [[1], [0, 5, 0], [128, 1, 127, 129], [0, 0, 300, 33, 0, 7], [513]]


@pytest.mark.parametrize("counts", SEGMENTS)
@pytest.mark.parametrize("K", [32, 96, 288])
@pytest.mark.parametrize("f32", [False, True])
def test_quantize_cols(gpu_lib, counts, K, f32):
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    src = wide((max(R // 2, 1), K), K)
    idx = synth.rng(3).integers(0, len(src), R).astype(np.int32)
    put = dev_f32 if f32 else dev_bf16
    po = gpu_lib.mx_padded_offsets(dev_i32(off))
    ref_po = M.padded_offsets(off)
    assert np.array_equal(host(po), ref_po)
    P = int(ref_po[-1])
    seg = dict(nseg=len(counts), seg_offsets=dev_i32(off), seg_padded_offsets=po)
    for gathered in (True, False):
        x = src[idx]
        t, ri = (put(src), dev_i32(idx)) if gathered else (put(x), None)
        for layout in (gpu_lib.NV4_COLS, gpu_lib.NV4_ROWS_AND_COLS):
            q = gpu_lib.MXFP4.empty(K, gpu_lib.mx_cols_capacity(R, len(counts)))
            q.codes.fill_(0xAA)
            q.scales.fill_(0xAA)
            gpu_lib.mxfp4_quantize(t, layout=layout, row_index=ri, out=q, **seg)
            c, b = M.quantize(M.by_segment(x, off))
            gc, gb = unpacked(q)
            assert np.array_equal(gc[:, :P], c) and np.array_equal(gb[:, :P // 32], b)
            # behind the last segment nothing is written
            assert (host(q.codes)[:, P // 2:] == 0xAA).all() and (gb[:, P // 32:] == 0xAA).all()
            if layout == gpu_lib.NV4_ROWS_AND_COLS:
                check_codes(q.rows_out, x)


@pytest.mark.parametrize("nseg", [257, 1000, 70000])
def test_quantize_cols_many_segments(gpu_lib, nseg):
    """Most of them empty, more than one and two passes of a workgroup's search; and rows behind
    the last segment, which neither direction writes."""
    r = synth.rng(nseg)
    counts = np.zeros(nseg, np.int64)
    counts[r.choice(nseg, 40, replace=False)] = r.integers(1, 300, 40)
    counts[[0, nseg - 1]] = [0, 5]
    off, K = np.concatenate([[0], np.cumsum(counts)]), 96
    R, extra = int(off[-1]), 70
    x = wide((R + extra, K), 7)
    po = M.padded_offsets(off)
    P = int(po[-1])
    if nseg <= 1024:
        assert np.array_equal(host(gpu_lib.mx_padded_offsets(dev_i32(off))), po)
    c, b = M.quantize(M.by_segment(x, off))
    for layout in (gpu_lib.NV4_COLS, gpu_lib.NV4_ROWS_AND_COLS):
        rows_out = None
        if layout == gpu_lib.NV4_ROWS_AND_COLS:
            rows_out = gpu_lib.MXFP4.empty(R + extra, K)
            rows_out.codes.fill_(0xAA)
            rows_out.scales.fill_(0xAA)
        q = gpu_lib.mxfp4_quantize(dev_bf16(x), layout=layout, nseg=nseg, seg_offsets=dev_i32(off),
                                   seg_padded_offsets=dev_i32(po), out_rows=rows_out)
        gc, gb = Q.unpack_codes(host(q.codes[:, :P // 2])), host(q.scales[:, :P // 32])
        assert np.array_equal(gc, c) and np.array_equal(gb, b)
        if rows_out is not None:
            check_codes(gpu_lib.MXFP4(rows_out.codes[:R], rows_out.scales[:R], R, K), x[:R])
            assert (rows_out.codes[R:] == 0xAA).all() and (rows_out.scales[R:] == 0xAA).all()


def test_offsets_behind_32_bits(gpu_lib):
    """More than 2^32 bytes of every large operand but the codes: the last rows against a call with
    those rows alone."""
    K, rows, tail = 2048, (1 << 20) + 4096 + 77, 300
    x = torch.randn(rows, K, device="cuda", dtype=torch.bfloat16)
    q, t = gpu_lib.mxfp4_quantize(x), gpu_lib.mxfp4_quantize(x[-tail:])
    assert x.numel() * 2 > 1 << 32 and same_bits(q.codes[-tail:], t.codes) and same_bits(q.scales[-tail:], t.scales)
    f32 = gpu_lib.mxfp4_dequantize(q, torch.float32)
    assert torch.equal(f32[-tail:], gpu_lib.mxfp4_dequantize(t, torch.float32))
    off = dev_i32(np.array([0, rows - tail, rows]))
    po = gpu_lib.mx_padded_offsets(off)
    seg = dict(layout=gpu_lib.NV4_ROWS_AND_COLS, nseg=2, seg_offsets=off, seg_padded_offsets=po)
    one = dev_i32(np.array([0, tail]))
    ref = gpu_lib.mxfp4_quantize(x[-tail:], layout=gpu_lib.NV4_COLS, nseg=1, seg_offsets=one,
                                 seg_padded_offsets=gpu_lib.mx_padded_offsets(one))
    for wide_x in (x, f32):
        c = gpu_lib.mxfp4_quantize(wide_x, **seg)
        start, end = po[1].item(), po[2].item()
        if wide_x is x:
            assert torch.equal(c.codes[:, start // 2:end // 2], ref.codes[:, :(end - start) // 2])
            assert torch.equal(c.scales[:, start // 32:end // 32], ref.scales[:, :(end - start) // 32])
        assert same_bits(c.rows_out.codes[-tail:], t.codes)
    del f32, c
    w = gpu_lib.mxfp4_quantize(torch.randn(2 * 2048, K, device="cuda", dtype=torch.bfloat16))
    y = gpu_lib.mxfp4_grouped_gemm(q, w, off, 2, 2048)
    ref = gpu_lib.mxfp4_grouped_gemm(t, gpu_lib.MXFP4(w.codes[2048:], w.scales[2048:], 2048, K), one, 1, 2048)
    # (other tiles may sum K in another order: at most K / 64 partial sums)
    assert y.numel() * 4 > 1 << 32
    assert ((y[-tail:] - ref).norm(dim=1) <= K / 64 * 2.0 ** -23 * 100 * ref.norm(dim=1)).all()


@pytest.mark.parametrize("nseg,m,K", [(1, 32, 32), (3, 96, 64), (2, 128, 160), (5, 288, 96)])
@pytest.mark.parametrize("f32", [False, True])
def test_quantize_cols_batched(gpu_lib, nseg, m, K, f32):
    x = wide((nseg * m, K), m)
    q = gpu_lib.mxfp4_quantize((dev_f32 if f32 else dev_bf16)(x), layout=gpu_lib.NV4_COLS_BATCHED, nseg=nseg)
    check_codes(q, x.reshape(nseg, m, K).transpose(0, 2, 1).reshape(nseg * K, m))


# ----------------------------------------------------------------------------- grouped GEMM

def check_product(got, A, B, off, E, N, swiglu=False):
    """FP32 results against FP64 on the same values, element by element."""
    n = 2 * N if swiglu else N
    raw = moe.grouped_gemm_m(A, B, off, E, n)
    tol = A.shape[1] * ULP * moe.grouped_gemm_m(np.abs(A), np.abs(B), off, E, n)
    ref = raw
    if swiglu:
        g, u, tg, tu = raw[:, :N], raw[:, N:], tol[:, :N], tol[:, N:]
        ref = moe.swiglu(raw)
        # |silu'| <= 1.1; exp2 and reciprocal of the hardware and three products: 2^-20 relative
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(ref) * 2.0 ** -20 + np.abs(g) * tu
    assert (np.abs(got - ref) <= tol + 1e-38).all(), float(np.max(np.abs(got - ref) / (tol + 1e-38)))
    return ref


COUNTS = [[5], [0, 1, 31, 33, 0], [64, 65, 127, 128, 129, 0], [300, 0, 257, 1, 520]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N", [(32, 8), (96, 33), (160, 256), (128, 1), (384, 288), (544, 130), (1056, 64)])
@pytest.mark.parametrize("epi", [0, 1])
def test_group_m(gpu_lib, counts, K, N, epi):
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R, n = int(off[-1]), N * (1 + epi)
    aq = gpu_lib.mxfp4_quantize(dev_bf16(synth.activations(R, K, K + N)))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * n, K), N)))
    C = torch.full((R + 3, N), 12345.0, dtype=torch.float32, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, epilogue=epi, C=C)
    check_product(host(C)[:R], vals(aq), vals(bq), off, E, N, swiglu=bool(epi))
    assert (host(C)[R:] == 12345.0).all()       # rows behind the last segment are left
    # BF16 is the FP32 result rounded to nearest even; the call repeats bitwise
    C16 = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, epilogue=epi, out_dtype=torch.bfloat16)
    assert np.array_equal(host(C16), bf16_rne_of(host(C)[:R]))
    again = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, epilogue=epi)
    assert same_bits(again, C[:R].contiguous())


@pytest.mark.parametrize("rule", [M.FLOOR, M.CEIL])
@pytest.mark.parametrize("N", [32, 96, 224, 768])
def test_swiglu_requantised_in_the_epilogue(gpu_lib, N, rule):
    counts = [130, 0, 77, 300]
    E, K, off = 4, 416, np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    aq = gpu_lib.mxfp4_quantize(dev_bf16(synth.activations(R, K, 1)))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * 2 * N, K), 2)))
    o = dict(M_cap=R, epilogue=gpu_lib.NV4_EPI_SWIGLU, rule=rule)
    plain = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, **o)
    for ct in (torch.float32, torch.bfloat16):
        q = gpu_lib.MXFP4.empty(R, N)
        q.scales.fill_(0xEE)
        C = torch.empty((R, N + 8), dtype=ct, device="cuda")[:, :N]
        gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, C=C, q_out=q, **o)
        assert same_bits(C.contiguous(), plain.to(ct))
        check_codes(q, host(plain), rule)
    alone = gpu_lib.MXFP4.empty(R, N)
    assert gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, q_out=alone, want_c=False, **o) is None
    assert same_bits(alone.codes, q.codes) and same_bits(alone.scales, q.scales)


def test_gather_is_the_materialised_gather(gpu_lib):
    counts, K, N, E = [70, 0, 300, 9], 320, 96, 4
    off = np.concatenate([[0], np.cumsum(counts)])
    R, T = int(off[-1]), 100
    x = synth.activations(T, K, 7)
    idx = synth.rng(8).integers(0, T, R).astype(np.int32)
    aq, ag = gpu_lib.mxfp4_quantize(dev_bf16(x)), gpu_lib.mxfp4_quantize(dev_bf16(x[idx]))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * N, K), 2)))
    one = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, a_rows=dev_i32(idx))
    two = gpu_lib.mxfp4_grouped_gemm(ag, bq, dev_i32(off), E, N, M_cap=R)
    assert same_bits(one, two)
    # rows outside A are clamped into it, and M_cap cuts the last rows off
    idx2 = idx.copy()
    idx2[:2] = [-9, T + 5]
    idx[:2] = [0, T - 1]
    out = torch.full((R, N), 7.0, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R - 5, a_rows=dev_i32(idx2), C=out)
    ref = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, a_rows=dev_i32(idx))
    assert same_bits(out[:R - 5].contiguous(), ref[:R - 5].contiguous()) and (out[R - 5:] == 7.0).all()


def test_nan_block_reaches_its_results_only(gpu_lib):
    x = synth.activations(40, 256, 1)
    x[3, 5] = np.nan
    aq = gpu_lib.mxfp4_quantize(dev_bf16(x))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((64, 256), 2)))
    C = host(gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(np.array([0, 40])), 1, 64))
    assert np.isnan(C[3]).all() and np.isfinite(np.delete(C, 3, 0)).all()


@pytest.mark.parametrize("counts", [[1], [0, 5, 0, 128], [300, 0, 129, 7, 0], [40, 1200, 3]])
@pytest.mark.parametrize("N,Mc", [(32, 32), (64, 288), (320, 96)])
def test_group_k(gpu_lib, counts, N, Mc):
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    a, b = synth.gradients((R, N), 4), synth.activations(R, Mc, 5)
    po = gpu_lib.mx_padded_offsets(dev_i32(off))
    cols = lambda t: gpu_lib.mxfp4_quantize(dev_bf16(t), layout=gpu_lib.NV4_COLS, nseg=E, seg_offsets=dev_i32(off),
                                            seg_padded_offsets=po)
    aq, bq = cols(a), cols(b)
    # NaN bytes behind the last segment must not matter
    rpo = M.padded_offsets(off)
    aq.scales[:, int(rpo[-1]) // 32:] = 255
    C = gpu_lib.mxfp4_grouped_gemm(aq, bq, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K)
    av, bv = M.rounded(M.by_segment(a, off)), M.rounded(M.by_segment(b, off))
    ref = moe.grouped_gemm_k(av, bv, rpo, E)
    tol = moe.grouped_gemm_k(np.abs(av), np.abs(bv), rpo, E) * ULP * (max(counts) + 128)
    assert (np.abs(host(C) - ref) <= tol).all()
    for e in range(E):
        if counts[e] == 0:
            assert (host(C)[e] == 0).all()
    C16 = gpu_lib.mxfp4_grouped_gemm(aq, bq, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=torch.bfloat16)
    assert np.array_equal(host(C16), bf16_rne_of(host(C)))


@pytest.mark.parametrize("N,ld,first", [(96, 96, 0), (96, 98, 1), (96, 97, 0), (95, 96, 0), (95, 95, 0), (352, 360, 3),
                                        (1, 1, 0), (2, 4, 2), (351, 352, 0)])
@pytest.mark.parametrize("epi", [0, 1])
@pytest.mark.parametrize("rows", [70, 900, 5000])
def test_bf16_results_of_any_alignment(gpu_lib, N, ld, first, epi, rows):
    """Every tile, column counts and row strides that do and do not allow stores of two columns:
    the BF16 rows are the FP32 rows rounded, and nothing else is written."""
    E, K = 2, 160
    off = dev_i32(np.array([0, rows // 3, rows - 2]))
    a = random_mx(gpu_lib, rows, K)
    b = random_mx(gpu_lib, E * N * (1 + epi), K)
    f32 = gpu_lib.mxfp4_grouped_gemm(a, b, off, E, N, M_cap=rows, epilogue=epi)
    buf = torch.full((rows, ld + first), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(a, b, off, E, N, M_cap=rows, epilogue=epi, C=buf[:, first:first + N])
    assert same_bits(buf[:rows - 2, first:first + N].contiguous(), f32[:rows - 2].bfloat16())
    assert (buf[:, :first] == 9).all() and (buf[:, first + N:] == 9).all() and (buf[rows - 2:] == 9).all()


def test_many_experts_and_tiles(gpu_lib):
    """More tiles than workgroups, uneven experts, 1024 experts."""
    for E, R, K, N in ((1024, 5000, 64, 40), (16, 20000, 256, 520)):
        r = synth.rng(E)
        counts = r.multinomial(R, r.dirichlet(np.full(E, 0.3)))
        off = np.concatenate([[0], np.cumsum(counts)])
        aq = gpu_lib.mxfp4_quantize(dev_bf16(synth.activations(R, K, 1)))
        bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * N, K), 2)))
        C = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N)
        check_product(host(C), vals(aq), vals(bq), off, E, N)


# ----------------------------------------------------------------------------- gradients

def lossless(shape, seed, scale=1.0):
    """Values every MXFP4 quantisation of which, in either direction, is exact: each block holds
    the largest code, every other value is a code under that scale."""
    v = synth.rng(seed).choice(np.array([-6, -4, -3, -2, -1, -.5, 0, .5, 1, 2, 3, 4, 6]), shape)
    v[::32, :] = 6
    v[:, ::32] = -6
    return (v * scale).astype(np.float32)


def test_linear_gradients_against_formula_and_differences(gpu_lib):
    """y = x W^T per expert.  On operands that quantise exactly the gradients are the formula's,
    and, y being linear, a difference quotient of sum(dy * y) over a whole entry of x or W is
    the gradient itself."""
    counts, K, N, E = [64, 0, 160, 32], 96, 64, 4
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    x, dy, W = lossless((R, K), 1), lossless((R, N), 2, 0.25), lossless((E * N, K), 3, 0.5)
    seg_of = np.repeat(np.arange(E), counts)
    po = gpu_lib.mx_padded_offsets(dev_i32(off))
    seg = dict(nseg=E, seg_offsets=dev_i32(off), seg_padded_offsets=po)
    dyc = gpu_lib.mxfp4_quantize(dev_bf16(dy), layout=gpu_lib.NV4_ROWS_AND_COLS, **seg)
    xc = gpu_lib.mxfp4_quantize(dev_bf16(x), layout=gpu_lib.NV4_COLS, **seg)
    wt = gpu_lib.mxfp4_quantize(dev_bf16(W), layout=gpu_lib.NV4_COLS_BATCHED, nseg=E)
    dx = host(gpu_lib.mxfp4_grouped_gemm(dyc.rows_out, wt, dev_i32(off), E, K)).astype(np.float64)
    dw = host(gpu_lib.mxfp4_grouped_gemm(dyc, xc, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K)).astype(np.float64)
    W3 = W.reshape(E, N, K).astype(np.float64)
    # every product and sum is a small multiple of 2^-4: exact in FP32
    assert np.array_equal(dx, np.einsum("rn,rnk->rk", dy.astype(np.float64), W3[seg_of]))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        assert np.array_equal(dw[e], dy[s].astype(np.float64).T @ x[s].astype(np.float64))

    def loss(xv, wv):
        y = gpu_lib.mxfp4_grouped_gemm(gpu_lib.mxfp4_quantize(dev_bf16(xv)), gpu_lib.mxfp4_quantize(dev_bf16(wv)),
                                       dev_i32(off), E, N)
        return float((host(y).astype(np.float64) * dy).sum())

    base = loss(x, W)
    r = synth.rng(4)
    for _ in range(6):
        i, j = int(r.integers(R)), int(r.integers(K))
        if x[i, j] not in (6, -6):
            x2 = x.copy()
            x2[i, j] = 0 if x[i, j] else 2
            assert loss(x2, W) - base == dx[i, j] * (x2[i, j] - x[i, j])
        i, j = int(r.integers(E * N)), int(r.integers(K))
        if W[i, j] not in (3, -3):
            W2 = W.copy()
            W2[i, j] = 0 if W[i, j] else 0.5
            assert loss(x, W2) - base == dw.reshape(E * N, K)[i, j] * (W2[i, j] - W[i, j])


# ----------------------------------------------------------------------------- the layer

def test_layer_forward_and_backward_stage_by_stage(gpu_lib):
    """mx_moe_forward and mx_moe_backward as they are used together: every stage on the GPU's
    own inputs, and the quantised SwiGLU rows from the epilogue."""
    cfg = synth.CONFIGS["tiny"]
    d = synth.layer_inputs(cfg, with_grads=True)
    W13, W2 = dev_bf16(d["W13"]), dev_bf16(d["W2"])
    w, wt = gpu_lib.mx_quantize_expert_weights(W13, W2), gpu_lib.mx_quantize_expert_weights_t(W13, W2)
    f = gpu_lib.mx_alloc_forward(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I, keep_hact=True, out_dtype=torch.float32)
    x = dev_bf16(d["X"])
    gpu_lib.mx_moe_forward(x, dev_f32(d["logits"]), w, cfg.k, f)
    ids, wts = moe.route_topk(d["logits"], cfg.k)
    p = moe.permute(ids, cfg.E)
    off, R = p["offsets"], cfg.R
    check_codes(f.xq, d["X"])
    check_codes(w.w13, d["W13"].reshape(-1, cfg.H))
    check_codes(wt.w2t, d["W2"].transpose(0, 2, 1).reshape(-1, cfg.H))
    assert np.array_equal(host(f.routing.row_token), p["row_token"])
    h32 = gpu_lib.mxfp4_grouped_gemm(f.xq, w.w13, f.routing.offsets, cfg.E, cfg.I, M_cap=R, a_rows=f.routing.row_token,
                                     epilogue=gpu_lib.NV4_EPI_SWIGLU)
    check_product(host(h32), vals(f.xq)[p["row_token"]], vals(w.w13), off, cfg.E, cfg.I, swiglu=True)
    check_codes(f.hq, host(h32))
    assert np.array_equal(host(f.hact), bf16_rne_of(host(h32)))
    check_product(host(f.y), vals(f.hq), vals(w.w2), off, cfg.E, cfg.H)
    ref = moe.combine(host(f.y), p["token_row"], wts)
    assert rel_frob(host(f.out), ref) <= 1e-5
    g = gpu_lib.mx_alloc_backward(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I, dgrad_dtype=torch.float32)
    gpu_lib.mx_moe_backward(x, f, wt, dev_bf16(d["dY2"]), dev_bf16(d["dY13"]), g)
    check_codes(g.dy2q, d["dY2"])
    check_codes(g.dy13q, d["dY13"])
    check_product(host(g.dhact), vals(g.dy2q), vals(wt.w2t), off, cfg.E, cfg.I)
    check_product(host(g.dxperm), vals(g.dy13q), vals(wt.w13t), off, cfg.E, cfg.H)
    po = M.padded_offsets(off)
    P = int(po[-1])
    col = lambda q: vals(q)[:, :P]
    for q, t in ((g.dy2c, d["dY2"]), (g.hc, host(f.hact)), (g.dy13c, d["dY13"]), (g.xc, d["X"][p["row_token"]])):
        assert np.array_equal(col(q), M.rounded(M.by_segment(np.asarray(t, np.float64), off)))
    for got, a, b in ((g.dw2, g.dy2c, g.hc), (g.dw13, g.dy13c, g.xc)):
        ref = moe.grouped_gemm_k(col(a), col(b), po, cfg.E)
        tol = moe.grouped_gemm_k(np.abs(col(a)), np.abs(col(b)), po, cfg.E) * ULP * (np.diff(po).max())
        assert (np.abs(host(got) - ref) <= tol).all()
    with pytest.raises(ValueError, match="keep_hact"):
        gpu_lib.mx_moe_backward(x, gpu_lib.mx_moe_forward(x, dev_f32(d["logits"]), w, cfg.k), wt, None, None)


# ----------------------------------------------------------------------------- a few tokens

def few_reference(x, ids, wts, w13v, w2v, rule=M.FLOOR):
    """Oracle output and how far an FP32 computation may be from it: sums as above, plus, for
    every SwiGLU value whose FP32 error can reach a rounding border, the step it may take."""
    out, h, gu, ab = M.layer(x, ids, wts, w13v, w2v, rule)
    T, k, I = h.shape
    g, u = gu[..., :I], gu[..., I:]
    dg, du = x.shape[1] * ULP * ab[..., :I], x.shape[1] * ULP * ab[..., I:]
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + np.abs(h) * 2.0 ** -20
    hb, db = h.reshape(T, k, -1, 32), dh.reshape(T, k, -1, 32)
    q0 = M.rounded(h, rule)
    move = np.zeros_like(h)
    amax = np.abs(hb).max(-1)
    reach = np.max(np.abs(hb) + db, -1), np.maximum(np.max(np.abs(hb) - db, -1), 0)
    for b in {0, -1, 1}:  # the block's exponent, or the neighbour an error can reach
        byte = M.scale_bytes(amax, rule).astype(int) + b
        ok = (byte <= M.scale_bytes(reach[0], rule)) & (byte >= M.scale_bytes(reach[1], rule))
        s = np.ldexp(1.0, byte - 127)[..., None]
        from oracle import formats as F
        enc = lambda v: F.e2m1_decode(F.e2m1_encode(np.clip(v / s, -8, 8).astype(np.float32))) * s
        far = np.maximum(np.abs(enc(hb + db) - q0.reshape(hb.shape)), np.abs(enc(hb - db) - q0.reshape(hb.shape)))
        move = np.maximum(move, np.where(ok[..., None], far, 0).reshape(h.shape))
    tol = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            W = np.abs(w2v[ids[t, j]])
            tol[t] += wts[t, j] * (W @ move[t, j] + (I + 64 * k) * ULP * (W @ np.abs(q0[t, j])))
    return out, tol + np.abs(out) * 2.0 ** -20


def few_case(gpu_lib, T, E, k, H, I, seed=0, rule=M.FLOOR):
    x = synth.activations(T, H, seed + 1)
    W13, W2 = synth.weights((E, 2 * I, H), seed + 2), synth.weights((E, H, I), seed + 3)
    lg = synth.logits_softmax(T, E, seed + 4)
    w = gpu_lib.mx_quantize_expert_weights(dev_bf16(W13), dev_bf16(W2), rule=rule)
    return x, lg, w, vals(w.w13).reshape(E, 2 * I, H), vals(w.w2).reshape(E, H, I)


@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 8, 2, 64, 32), (1, 2, 1, 32, 32), (2, 40, 3, 96, 160), (5, 16, 8, 160, 64), (16, 4, 2, 288, 96),
    (17, 3, 3, 128, 224), (33, 130, 6, 64, 64), (64, 8, 2, 544, 288), (64, 2, 2, 1056, 32), (7, 300, 32, 64, 32),
    (64, 1, 1, 64, 64), (3, 1024, 4, 32, 32), (9, 520, 2, 2080, 32),
    (2, 8, 8, 64, 1056), (8, 2, 2, 64, 32), (4, 4, 4, 4128, 32), (3, 64, 4, 32, 800)])
def test_few(gpu_lib, T, E, k, H, I):
    for rule, flags in ((M.FLOOR, 0), (M.CEIL, gpu_lib.NV4_RENORM)):
        x, lg, w, v13, v2 = few_case(gpu_lib, T, E, k, H, I, seed=T + H, rule=rule)
        ids, wts = moe.route_topk(lg, k, renorm=bool(flags))
        gi = torch.empty((T, k), dtype=torch.int32, device="cuda")
        gw = torch.empty((T, k), dtype=torch.float32, device="cuda")
        o = dict(flags=flags, rule=rule)
        out = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, topk_ids=gi, topk_w=gw, out_dtype=torch.float32, **o)
        assert np.array_equal(host(gi), ids)
        rt = gpu_lib.moe_permute(dev_f32(lg), E, k, flags=flags)
        assert same_bits(gw, rt.topk_w)
        ref, tol = few_reference(x, ids, host(gw).astype(np.float64), v13, v2, rule)
        assert (np.abs(host(out) - ref) <= tol + 1e-38).all(), float(np.max(np.abs(host(out) - ref) / (tol + 1e-38)))
        assert rel_frob(host(gw), wts) <= 1e-6
        # BF16 and FP32 inputs and outputs agree; given routing gives the same bits
        o16 = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, **o)
        assert np.array_equal(host(o16), bf16_rne_of(host(out)))
        assert same_bits(gpu_lib.mx_moe_few(dev_f32(x), dev_f32(lg), w, k, **o), o16)
        given = gpu_lib.mx_moe_few(dev_bf16(x), None, w, k, topk_ids=gi, topk_w=gw, rule=rule, out_dtype=torch.float32)
        assert same_bits(given, out)


def test_few_is_the_composed_layer(gpu_lib):
    """At the decode shape: the same layer as mx_moe_forward up to the codes that the order of
    the FP32 sums moves.  Each moved code changes a SwiGLU value by at most half of it, so with
    at most 0.3 such values in a row of k * I the rows differ by 0.5 sqrt(0.3 / (k I)) < 5e-3 of
    their norm."""
    T, E, k, H, I = 64, 32, 8, 2048, 768
    x, lg, w, *_ = few_case(gpu_lib, T, E, k, H, I, seed=11)
    bufs = gpu_lib.mx_alloc_forward(T, H, E, k, I, out_dtype=torch.float32)
    gpu_lib.mx_moe_forward(dev_bf16(x), dev_f32(lg), w, k, bufs)
    out = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, out_dtype=torch.float32)
    assert rel_frob(host(out), host(bufs.out).astype(np.float64)) <= 5e-3
    # a token alone is the token in the batch
    one = gpu_lib.mx_moe_few(dev_bf16(x[9:10]), dev_f32(lg[9:10]), w, k, out_dtype=torch.float32)
    assert rel_frob(host(one)[0], host(out)[9].astype(np.float64)) <= 5e-3


def test_few_odd_routing(gpu_lib):
    T, E, k, H, I = 6, 5, 3, 96, 64
    x, lg, w, v13, v2 = few_case(gpu_lib, T, E, k, H, I)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = np.array([[0, 0, 0], [1, 4, 1], [2, 3, 4], [7, 1, -1], [-3, 9, 5], [4, 4, 2]], np.int32)
    wts = synth.rng(1).random((T, k)).astype(np.float32)
    out = gpu_lib.mx_moe_few(dev_bf16(x), None, w, k, topk_ids=dev_i32(ids), topk_w=dev_f32(wts),
                             out_dtype=torch.float32, dev_status=st)
    assert st.item() == gpu_lib.NV4_DS_BAD_EXPERT
    bad = (ids < 0) | (ids >= E)
    ref, tol = few_reference(x, np.where(bad, 0, ids), np.where(bad, 0, wts).astype(np.float64), v13, v2)
    assert (np.abs(host(out) - ref) <= tol + 1e-38).all() and (host(out)[4] == 0).all()
    # logits: ties go to the lower id; a token without a number routes nowhere
    tied = np.zeros((T, E), np.float32)
    tied[2] = -np.inf
    tied[2, 3] = 1.0
    tied[5] = np.nan
    st.zero_()
    gi = torch.empty((T, k), dtype=torch.int32, device="cuda")
    out = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(tied), w, k, topk_ids=gi, out_dtype=torch.float32, dev_status=st)
    assert st.item() == gpu_lib.NV4_DS_NAN_LOGIT
    assert (host(gi)[[0, 1, 3, 4]] == [0, 1, 2]).all() and (host(gi)[2] == [3, 0, 1]).all()
    assert (host(out)[5] == 0).all() and np.isfinite(host(out)).all()
    assert rel_frob(host(out)[2], M.layer(x[2:3], np.array([[3]]), np.ones((1, 1)), v13, v2)[0][0]) <= 0.05


def test_few_strides_nan_and_rows_left(gpu_lib):
    T, E, k, H, I = 5, 4, 2, 128, 64
    x, lg, w, *_ = few_case(gpu_lib, T, E, k, H, I)
    ref = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k)
    wide_x = torch.full((T, H + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_x[:, 8:8 + H] = dev_bf16(x)
    buf = torch.full((T + 2, H + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.mx_moe_few(wide_x[:, 8:8 + H], dev_f32(lg), w, k, out=buf[1:T + 1, 3:3 + H])
    assert same_bits(buf[1:T + 1, 3:3 + H].contiguous(), ref)
    assert (buf[0] == 9).all() and (buf[T + 1] == 9).all() and (buf[:, :3] == 9).all() and (buf[:, 3 + H:] == 9).all()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x[2, 70] = np.inf
    out = host(gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, dev_status=st))
    assert st.item() == gpu_lib.NV4_DS_NONFINITE
    assert np.isnan(out[2]).all() and np.array_equal(np.delete(out, 2, 0), np.delete(host(ref), 2, 0))
    for bad in (dict(topk_w=torch.zeros(3, device="cuda")), dict(out=torch.empty(T, H + 1, device="cuda")),
                dict(ws=torch.empty(16, device="cuda")), dict(topk_ids=torch.zeros(T, k, device="cuda"))):
        with pytest.raises(ValueError):
            gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, **bad)
    with pytest.raises(gpu_lib.NV4Error):
        gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(lg), w, k, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    empty = gpu_lib.mx_moe_few(dev_bf16(x)[:0], dev_f32(lg)[:0], w, k)
    assert empty.shape == (0, H)


@pytest.mark.parametrize("T,E,k,H,I", [
    (64, 3, 2, 96, 1632), (40, 6, 2, 64, 1632), (36, 2, 2, 4128, 32), (24, 3, 3, 2112, 64), (1, 6, 3, 64, 3136),
    (25, 9, 3, 32, 800), (64, 90, 1, 64, 64)])
def test_few_many_rows_and_windows(gpu_lib, T, E, k, H, I):
    """More than 16 rows of an expert, and more of either matrix's K than a wave holds at once."""
    test_few(gpu_lib, T, E, k, H, I)


@pytest.mark.parametrize("T,E,k,H,I", [
    (12, 260, 8, 64, 32), (16, 300, 8, 96, 64), (64, 256, 2, 64, 32), (13, 128, 8, 64, 32), (12, 128, 8, 64, 32),
    (16, 8, 2, 64, 96), (17, 8, 2, 64, 96), (2, 600, 32, 64, 32), (4, 1024, 32, 64, 32)])
def test_few_on_either_side_of_its_rule(gpu_lib, T, E, k, H, I):
    test_few(gpu_lib, T, E, k, H, I)


def random_mx(gpu_lib, rows, K):
    """Random codes under scales 2^-7 .. 1, made on the GPU."""
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((rows, gpu_lib.mxfp4_scale_stride(K)), dtype=torch.uint8, device="cuda")
    scales[:, :K // 32] = torch.randint(120, 128, (rows, K // 32), dtype=torch.uint8, device="cuda")
    return gpu_lib.MXFP4(codes, scales, rows, K)


def test_few_more_experts_than_a_pass_holds(gpu_lib):
    """1024 experts in use and one workgroup a column tile.  The whole is the sum of its quarters:
    FP32 sums of 32 terms in another order, each off by at most 32 2^-24 of the terms' sum."""
    T, E, k, H, I = 64, 1024, 32, 2080, 32
    w = gpu_lib.MXExpertWeights(random_mx(gpu_lib, E * 2 * I, H), random_mx(gpu_lib, E * H, I), E, H, I)
    x = torch.randn(T, H, device="cuda")
    ids = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(T // 2)]).int()
    ids = torch.cat([torch.arange(T // 2 * k, device="cuda").reshape(T // 2, k).int() % E, ids])  # every expert
    wts = torch.rand(T, k, device="cuda") + 0.1
    o = dict(out_dtype=torch.float32)
    out = gpu_lib.mx_moe_few(x, None, w, k, topk_ids=ids, topk_w=wts, **o)
    part = [gpu_lib.mx_moe_few(x, None, w, 8, topk_ids=ids[:, i:i + 8].contiguous(),
                               topk_w=wts[:, i:i + 8].contiguous(), **o).double() for i in range(0, k, 8)]
    size = sum(p.abs() for p in part)
    assert torch.unique(ids).numel() == E and size.min() > 0
    assert ((out.double() - sum(part)).norm() / sum(part).norm()).item() <= 32 * 2.0 ** -24 * 4


def test_weights_above_4_gib(gpu_lib):
    """Experts on either side of 4 GiB of codes against the same two experts alone.  FP32 sums of
    K / 64 partial sums, possibly by other tiles: off by at most K / 64 2^-24 of the terms' sum,
    of which a random row's norm is at least a hundredth."""
    E, H, I = 132, 8192, 4096
    w13, w2 = random_mx(gpu_lib, E * 2 * I, H), random_mx(gpu_lib, E * H, I)
    assert w13.codes.numel() > 1 << 32
    pick = lambda m, n: gpu_lib.MXFP4(*(torch.cat([t[:n], t[-n:]]) for t in (m.codes, m.scales)), 2 * n, m.K)
    two13, two2 = pick(w13, 2 * I), pick(w2, H)
    R = 80
    x = gpu_lib.mxfp4_quantize(torch.randn(R, H, device="cuda", dtype=torch.bfloat16))
    far = torch.tensor([0] + [35] * (E - 1) + [R], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, 35, R], dtype=torch.int32, device="cuda")
    f32 = dict(out_dtype=torch.float32)
    got = gpu_lib.mxfp4_grouped_gemm(x, w13, far, E, 2 * I, M_cap=R, **f32)
    ref = gpu_lib.mxfp4_grouped_gemm(x, two13, near, 2, 2 * I, M_cap=R, **f32)
    tol = H / 64 * 2.0 ** -24 * 100
    assert ((got - ref).norm(dim=1) <= tol * ref.norm(dim=1)).all() and ref.abs().max() > 0
    xf = torch.randn(R // 2, H, device="cuda", dtype=torch.bfloat16)
    wts = torch.rand(R // 2, 2, device="cuda")
    for T in (1, 20, 40):  # each of the three ways through the layer
        ids = torch.tensor([[E - 1, 0]], dtype=torch.int32, device="cuda").repeat(T, 1)
        few = lambda m13, m2, n, ids: gpu_lib.mx_moe_few(xf[:T], None, gpu_lib.MXExpertWeights(m13, m2, n, H, I), 2,
                                                         topk_ids=ids, topk_w=wts[:T].contiguous(), **f32)
        got, ref = few(w13, w2, E, ids), few(two13, two2, 2, (ids > 0).int())
        # (a sum next to a rounding border may take the other code: 0.3 of them in a row of 2 I)
        assert ((got - ref).norm(dim=1) <= 5e-3 * ref.norm(dim=1)).all() and ref.abs().max() > 0


# ----------------------------------------------------------------------------- streams and graphs

def test_side_stream_and_two_calls_at_once(gpu_lib):
    T, E, k, H, I = 33, 16, 4, 512, 256
    x, lg, w, *_ = few_case(gpu_lib, T, E, k, H, I)
    xd, ld = dev_bf16(x), dev_f32(lg)
    ref_few = gpu_lib.mx_moe_few(xd, ld, w, k)
    ref = gpu_lib.mx_moe_forward(xd, ld, w, k).out.clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append((gpu_lib.mx_moe_few(xd, ld, w, k, stream=s1), ref_few))
        outs.append((gpu_lib.mx_moe_few(xd, ld, w, k, stream=s2), ref_few))
        with torch.cuda.stream(s2):
            outs.append((gpu_lib.mx_moe_forward(xd, ld, w, k).out, ref))
    torch.cuda.synchronize()
    for got, want in outs:
        assert same_bits(got, want)


def test_graphs_that_share_a_workspace(gpu_lib):
    """Two captured batches of different sizes and an eager one in one workspace, in turn."""
    E, k, H, I = 24, 4, 544, 96
    x, lg, w, *_ = few_case(gpu_lib, 64, E, k, H, I)
    xd, ld = dev_bf16(x), dev_f32(lg)
    ws = torch.empty(gpu_lib.load().mx_moe_few_workspace(64, E, k, H, I), dtype=torch.uint8, device="cuda")
    want = {T: gpu_lib.mx_moe_few(xd[:T], ld[:T], w, k) for T in (1, 2, 9, 30, 64)}
    out = {T: torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for T in want}
    graphs = {}
    for T in want:
        graphs[T] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[T]):
            gpu_lib.mx_moe_few(xd[:T], ld[:T], w, k, ws=ws, out=out[T])
    for T in (64, 1, 9, 64, 2, 30, 1, 64, 9, 30, 2):
        out[T].zero_()
        ws.fill_(0xFF)
        graphs[T].replay()
        got = gpu_lib.mx_moe_few(xd[:30], ld[:30], w, k, ws=ws)
        torch.cuda.synchronize()
        assert same_bits(out[T], want[T]) and same_bits(got, want[30])


def test_empty_batches(gpu_lib):
    E, k, H, I = 6, 2, 64, 32
    x, lg, w, *_ = few_case(gpu_lib, 3, E, k, H, I)
    assert gpu_lib.mx_moe_few(dev_bf16(x)[:0], dev_f32(lg)[:0], w, k).shape == (0, H)
    q = gpu_lib.mxfp4_quantize(dev_bf16(x)[:0])
    assert q.codes.shape == (0, H // 2) and gpu_lib.mxfp4_dequantize(q).shape == (0, H)
    zero = dev_i32(np.zeros(E + 1))
    po = gpu_lib.mx_padded_offsets(zero)
    assert (po == 0).all()
    # rows, but none in a segment: nothing is written; weight gradients of empty ranges are zeros
    c = gpu_lib.MXFP4.empty(H, gpu_lib.mx_cols_capacity(3, E))
    c.codes.fill_(0xAA)
    c.scales.fill_(0xAA)
    gpu_lib.mxfp4_quantize(dev_bf16(x), layout=gpu_lib.NV4_COLS, nseg=E, seg_offsets=zero, seg_padded_offsets=po, out=c)
    assert (c.codes == 0xAA).all() and (c.scales == 0xAA).all()
    dw = gpu_lib.mxfp4_grouped_gemm(c, c, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K)
    assert dw.shape == (E, H, H) and (dw == 0).all()
    y = torch.full((3, 2 * I), 7.0, device="cuda")
    gpu_lib.mxfp4_grouped_gemm(gpu_lib.mxfp4_quantize(dev_bf16(x)), w.w13, zero, E, 2 * I, C=y)
    assert (y == 7).all()


def test_captured_and_replayed(gpu_lib):
    """Forward, backward and the few-token layer in one graph, replayed with changed inputs
    between eager calls: every replay equals the eager result."""
    cfg = synth.CONFIGS["tiny"]
    d = synth.layer_inputs(cfg, with_grads=True)
    W13, W2 = dev_bf16(d["W13"]), dev_bf16(d["W2"])
    w, wt = gpu_lib.mx_quantize_expert_weights(W13, W2), gpu_lib.mx_quantize_expert_weights_t(W13, W2)
    dY2, dY13 = dev_bf16(d["dY2"]), dev_bf16(d["dY13"])
    x, lg = dev_bf16(d["X"]), dev_f32(d["logits"])
    alloc = lambda: (gpu_lib.mx_alloc_forward(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I, keep_hact=True),
                     gpu_lib.mx_alloc_backward(cfg.T, cfg.H, cfg.E, cfg.k, cfg.I),
                     torch.empty((20, cfg.H), dtype=torch.bfloat16, device="cuda"),
                     torch.empty(gpu_lib.load().mx_moe_few_workspace(20, cfg.E, cfg.k, cfg.H, cfg.I), dtype=torch.uint8,
                                 device="cuda"))

    def step(f, g, few, ws):
        gpu_lib.mx_moe_forward(x, lg, w, cfg.k, f)
        gpu_lib.mx_moe_backward(x, f, wt, dY2, dY13, g)
        gpu_lib.mx_moe_few(x[:20], lg[:20], w, cfg.k, out=few, ws=ws)
        return f.out, g.dhact, g.dxperm, g.dw2, g.dw13, few

    eager, captured = alloc(), alloc()
    step(*captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*captured)
    for i in range(3):
        x.copy_(dev_bf16(synth.activations(cfg.T, cfg.H, 100 + i)))
        lg.copy_(dev_f32(synth.logits_softmax(cfg.T, cfg.E, 200 + i)))
        want = [t.clone() for t in step(*eager)]
        torch.cuda.synchronize()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert same_bits(a, b)
