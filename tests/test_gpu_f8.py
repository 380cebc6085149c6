"""GPU FP8 calls against the oracle: codes and scales bit for bit; products within the rounding of
their FP32 sums; repeated calls bitwise equal."""

import numpy as np
import pytest
import torch

import synth
from oracle import formats as F
from oracle import fp8 as M
from oracle import moe
from oracle import mxfp4 as MX
from tests.gpu_util import dev_bf16, dev_f32, dev_i32, host, same_bits

pytestmark = pytest.mark.gpu

# An FP32 sum of n products is off by at most n - 1 roundings of partial sums, each at most
# 2^-24 of a partial sum of |products| when it rounds to nearest and 2^-23 when it truncates.
ULP = 2.0 ** -23
# BF16 results: the matrix instruction adds eight products at the exponent of the largest and cuts each of the
# others off 13 bits behind it: 7 cuts of at most 2^-13 of the largest product.
CUT = 7 * 2.0 ** -13
HALF_BF16 = 2.0 ** -8
RULES = [M.FP32, M.POW2]


def vals(q):
    """FP64 values of a row-scaled tensor."""
    return M.values(host(q.codes), host(q.scales).reshape(q.rows, -1))


def tile_vals(q):
    c, s = host(q.codes).reshape(q.nseg, -1, q.K), host(q.scales)
    return np.concatenate([M.tile_values(c[i], s[i]) for i in range(q.nseg)])


def same_floats(a, b):
    return np.array_equal(np.asarray(a, np.float32).view(np.uint32), np.asarray(b, np.float32).view(np.uint32))


def check_codes(q, x, rule=M.FP32):
    c, G = M.quantize(np.asarray(x, np.float32), rule)
    got = host(q.scales)
    assert same_floats(np.nan_to_num(got, nan=-1), np.nan_to_num(G, nan=-1)), "scales"
    assert np.array_equal(host(q.codes), c), "codes"
    assert q.rule == rule and q.nseg == 0


def wide(shape, seed):
    """Values over the whole range of exponents a gradient meets, zeros, empty blocks and ties among them."""
    r = synth.rng(seed)
    n = -(-shape[1] // 64)
    x = r.standard_normal(shape) * np.exp2(r.integers(-30, 20, (shape[0], n))).repeat(64, 1)[:, :shape[1]]
    x[r.random(shape) < 0.2] *= 0.0
    x[:, :128][r.random(shape[0]) < 0.1] = 0.0
    t = r.random(shape) < 0.2                       # three quarters and such of the row's largest: ties
    x = np.where(t, np.abs(x).max(1, keepdims=True) * r.choice([0.75, -0.375, 0.65625], shape), x)
    return synth.to_bf16_values(x.astype(np.float32))


# ----------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("rows,K", [(1, 16), (1, 2048), (3, 112), (33, 144), (257, 1040), (1025, 2048), (4, 16400)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rule", RULES)
def test_quantize_rows(gpu_lib, rows, K, f32, rule):
    x = wide((rows, K), rows + K)
    if f32:
        x = x * (1 + synth.rng(9).random((rows, K), dtype=np.float32) * np.float32(1e-3))
    q = gpu_lib.fp8_quantize(dev_f32(x) if f32 else dev_bf16(x), rule=rule)
    check_codes(q, x, rule)
    v = vals(q)
    d = gpu_lib.fp8_dequantize(q, torch.float32)
    assert same_floats(host(d), v)
    assert same_bits(gpu_lib.fp8_dequantize(q), d.bfloat16())


@pytest.mark.parametrize("rule", RULES)
def test_quantize_extremes(gpu_lib, rule):
    """Subnormal and largest blocks, negative zeros, NaN and infinity in a block."""
    x = np.zeros((9, 256), np.float32)
    x[0, :4] = [1e-45, -1e-45, 3e-45, 5e-44]
    x[1] = np.float32(9e-41)
    x[2, :3] = [3.4028235e38, -3.0e38, 1e38]
    x[3] = -0.0
    x[4, 3], x[5, 140], x[6, 2] = np.nan, np.inf, -np.inf
    x[4, 128:] = 1.0
    x[7, :5] = [1.1754944e-38, 2.3509887e-38, 4e-38, -6e-38, 1e-39]
    x[8, :3] = [5.2e-36, 5.3e-36, -1e-36]                       # 448 / 5.27e-36 is 2^126
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (dev_f32(x), dev_bf16(x)):
        st.zero_()
        q = gpu_lib.fp8_quantize(t, dev_status=st, rule=rule)
        check_codes(q, t.float().cpu().numpy(), rule)
        assert st.item() == gpu_lib.NV4_DS_NONFINITE
        d = host(gpu_lib.fp8_dequantize(q))
        assert np.isnan(d[4, :128]).all() and np.isnan(d[5, 128:]).all() and np.isnan(d[6, :128]).all()
        assert np.isfinite(d[4, 128:]).all()
        st.zero_()
        gpu_lib.fp8_quantize(t[:4], dev_status=st, rule=rule)
        # (FP32's largest value is BF16's infinity)
        assert st.item() == (0 if t.dtype == torch.float32 else gpu_lib.NV4_DS_NONFINITE)
        for layout in (gpu_lib.NV4_COLS, gpu_lib.NV4_ROWS_AND_COLS):
            st.zero_()
            off = dev_i32(np.array([0, 9]))
            qc = gpu_lib.fp8_quantize(t, layout=layout, seg_offsets=off, seg_padded_offsets=gpu_lib.mx_padded_offsets(off),
                                      dev_status=st, rule=rule)
            assert st.item() == gpu_lib.NV4_DS_NONFINITE
            c, G = M.quantize(np.pad(t.float().cpu().numpy(), ((0, 119), (0, 0))).T, rule)
            assert np.array_equal(host(qc.codes)[:, :128], c)
            assert same_floats(np.nan_to_num(host(qc.scales)[:, 0], nan=-1), np.nan_to_num(G[:, 0], nan=-1))
            if layout == gpu_lib.NV4_ROWS_AND_COLS:
                check_codes(qc.rows_out, t.float().cpu().numpy(), rule)


def test_every_positive_bf16_maximum(gpu_lib):
    """Each finite BF16 magnitude as a block's largest, with its ties."""
    a = (np.arange(1, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    x = np.zeros((len(a), 16), np.float32)
    x[:, 0] = a
    with np.errstate(under="ignore"):
        for i, f in enumerate([0.75, 0.375, -0.1875, 0.65625, 0.0009765625]):
            x[:, 1 + i] = synth.to_bf16_values(a * np.float32(f))
    for rule in RULES:
        q = gpu_lib.fp8_quantize(dev_bf16(x), rule=rule)
        check_codes(q, x, rule)
        top = F.e4m3_decode(host(q.codes)[:, 0])
        big = a >= 2.0 ** -117
        assert (top[big] > 223).all() and (rule == M.POW2 or (top[big] == 448).all())


def test_quantize_strided_and_gathered(gpu_lib):
    x = wide((40, 192), 5)
    big = dev_bf16(np.concatenate([x, x[:, :64]], 1))
    check_codes(gpu_lib.fp8_quantize(big[:, 64:176]), x[:, 64:176])
    idx = np.array([39, 0, 7, 7, 21], np.int32)
    check_codes(gpu_lib.fp8_quantize(dev_bf16(x), row_index=dev_i32(idx)), x[idx])
    # an index outside x reads its nearest row
    q = gpu_lib.fp8_quantize(dev_bf16(x), row_index=dev_i32(np.array([-5, 99])))
    check_codes(q, x[[0, 39]])


SEGMENTS = [[1], [0, 5, 0], [128, 1, 127, 129], [0, 0, 300, 33, 0, 7], [513]]


@pytest.mark.parametrize("counts", SEGMENTS)
@pytest.mark.parametrize("K", [16, 112, 288])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rule", RULES)
def test_quantize_cols(gpu_lib, counts, K, f32, rule):
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    src = wide((max(R // 2, 1), K), K)
    idx = synth.rng(3).integers(0, len(src), R).astype(np.int32)
    put = dev_f32 if f32 else dev_bf16
    po = gpu_lib.mx_padded_offsets(dev_i32(off))
    ref_po = MX.padded_offsets(off)
    P = int(ref_po[-1])
    seg = dict(nseg=len(counts), seg_offsets=dev_i32(off), seg_padded_offsets=po, rule=rule)
    for gathered in (True, False):
        x = src[idx]
        t, ri = (put(src), dev_i32(idx)) if gathered else (put(x), None)
        for layout in (gpu_lib.NV4_COLS, gpu_lib.NV4_ROWS_AND_COLS):
            q = gpu_lib.FP8.empty(K, gpu_lib.mx_cols_capacity(R, len(counts)))
            q.codes.fill_(0xAA)
            q.scales.fill_(7.0)
            gpu_lib.fp8_quantize(t, layout=layout, row_index=ri, out=q, **seg)
            c, G = M.quantize(MX.by_segment(x, off).astype(np.float32), rule)
            assert np.array_equal(host(q.codes)[:, :P], c) and same_floats(host(q.scales)[:, :P // 128], G)
            # behind the last segment nothing is written
            assert (host(q.codes)[:, P:] == 0xAA).all() and (host(q.scales)[:, P // 128:] == 7.0).all()
            if layout == gpu_lib.NV4_ROWS_AND_COLS:
                check_codes(q.rows_out, x, rule)


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
    po = MX.padded_offsets(off)
    P = int(po[-1])
    c, G = M.quantize(MX.by_segment(x, off).astype(np.float32))
    for f32 in (False, True):
        for layout in (gpu_lib.NV4_COLS, gpu_lib.NV4_ROWS_AND_COLS):
            rows_out = None
            if layout == gpu_lib.NV4_ROWS_AND_COLS:
                rows_out = gpu_lib.FP8.empty(R + extra, K)
                rows_out.codes.fill_(0xAA)
                rows_out.scales.fill_(7.0)
            q = gpu_lib.fp8_quantize((dev_f32 if f32 else dev_bf16)(x), layout=layout, nseg=nseg, seg_offsets=dev_i32(off),
                                     seg_padded_offsets=dev_i32(po), out_rows=rows_out)
            assert np.array_equal(host(q.codes[:, :P]), c) and same_floats(host(q.scales[:, :P // 128]), G)
            if rows_out is not None:
                check_codes(gpu_lib.FP8(rows_out.codes[:R], rows_out.scales[:R], R, K), x[:R])
                assert (rows_out.codes[R:] == 0xAA).all() and (rows_out.scales[R:] == 7.0).all()


@pytest.mark.parametrize("nseg,m,K", [(1, 16, 16), (3, 100, 64), (2, 128, 160), (5, 288, 272), (2, 1, 128)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rule", RULES)
def test_quantize_tiles_and_transpose(gpu_lib, nseg, m, K, f32, rule):
    x = wide((nseg * m, K + 16), m)
    t = (dev_f32 if f32 else dev_bf16)(x)[:, :K]
    x = x[:, :K]
    q = gpu_lib.fp8_quantize(t, layout=gpu_lib.NV4_F8_TILES, nseg=nseg, rule=rule)
    ref = [M.quantize_tiles(x[i * m:(i + 1) * m], rule) for i in range(nseg)]
    assert q.nseg == nseg and q.rule == rule
    assert np.array_equal(host(q.codes), np.concatenate([c for c, _ in ref]))
    assert same_floats(host(q.scales), np.stack([G for _, G in ref]))
    v = tile_vals(q)
    assert same_floats(host(gpu_lib.fp8_dequantize(q, torch.float32)), v)
    if m % 16:
        with pytest.raises(gpu_lib.NV4Error, match="NV4_EALIGN"):
            gpu_lib.fp8_transpose(q)
        return
    qt = gpu_lib.fp8_transpose(q)
    assert (qt.rows, qt.K, qt.nseg, qt.rule) == (nseg * K, m, nseg, rule)
    assert np.array_equal(host(qt.codes).reshape(nseg, K, m), host(q.codes).reshape(nseg, m, K).transpose(0, 2, 1))
    assert same_floats(host(qt.scales), host(q.scales).transpose(0, 2, 1))


def test_tiles_with_a_value_that_is_not_finite(gpu_lib):
    x = wide((256, 256), 1)
    x[130, 5] = np.inf
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = gpu_lib.fp8_quantize(dev_bf16(x), layout=gpu_lib.NV4_F8_TILES, dev_status=st)
    s = host(q.scales)[0]
    assert st.item() == gpu_lib.NV4_DS_NONFINITE and np.isnan(s[1, 0]) and np.isfinite(np.delete(s.ravel(), 2)).all()
    assert (host(q.codes)[128:, :128] == 0).all()


# ----------------------------------------------------------------------------- grouped GEMM

def check_product(got, A, B, off, E, N, swiglu=False, bf16=False):
    """Results against FP64 on the same values, element by element."""
    n = 2 * N if swiglu else N
    raw = moe.grouped_gemm_m(A, B, off, E, n)
    # K products, and for each block a rounding of its scale and one of its product
    tol = (A.shape[1] + 3 * (A.shape[1] // 128 + 1)) * ULP + (CUT if bf16 else 0)
    tol = tol * moe.grouped_gemm_m(np.abs(A), np.abs(B), off, E, n)
    ref = raw
    if swiglu:
        g, u, tg, tu = raw[:, :N], raw[:, N:], tol[:, :N], tol[:, N:]
        ref = moe.swiglu(raw)
        # |silu'| <= 1.1; the sigmoid's and the products' own error
        tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(ref) * (1.25 * np.abs(g) + 8) * 2.0 ** -24 + np.abs(g) * tu
    if bf16:
        tol = tol + HALF_BF16 * (np.abs(ref) + tol)
    assert (np.abs(got - ref) <= tol + 1e-38).all(), float(np.max(np.abs(got - ref) / (tol + 1e-38)))
    return ref


def weights(lib, E, n, K, seed, rule=M.FP32):
    return lib.fp8_quantize(dev_bf16(synth.weights((E * n, K), seed)), layout=lib.NV4_F8_TILES, nseg=E, rule=rule)


COUNTS = [[5], [0, 1, 31, 33, 0], [64, 65, 127, 128, 129, 0], [300, 0, 257, 1, 520]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,epi", [(16, 8, 0), (112, 33, 0), (160, 256, 0), (128, 1, 0), (400, 288, 0), (544, 130, 0),
                                     (1040, 64, 0), (144, 32, 1), (128, 96, 1), (528, 288, 1), (2048, 160, 1)])
@pytest.mark.parametrize("rule", RULES)
def test_group_m(gpu_lib, counts, K, N, epi, rule):
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R, n = int(off[-1]), N * (1 + epi)
    aq = gpu_lib.fp8_quantize(dev_bf16(synth.activations(R, K, K + N)), rule=rule)
    bq = weights(gpu_lib, E, n, K, N, rule)
    C = torch.full((R + 3, N), 12345.0, dtype=torch.float32, device="cuda")
    gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, epilogue=epi, C=C)
    check_product(host(C)[:R], vals(aq), tile_vals(bq), off, E, N, swiglu=bool(epi))
    assert (host(C)[R:] == 12345.0).all()       # rows behind the last segment are left
    C16 = torch.full((R + 3, N), 12345.0, dtype=torch.bfloat16, device="cuda")
    o = dict(M_cap=R, epilogue=epi)
    gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, C=C16, **o)
    check_product(host(C16)[:R], vals(aq), tile_vals(bq), off, E, N, swiglu=bool(epi), bf16=True)
    assert (C16[R:] == 12352.0).all()           # (12345 as BF16)
    # the calls repeat bitwise
    assert same_bits(gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, **o), C[:R].contiguous())
    assert same_bits(gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, out_dtype=torch.bfloat16, **o), C16[:R].contiguous())


def small_integers(shape, seed):
    """Codes whose products and sums every way of adding holds exactly: integers up to 8."""
    return synth.rng(seed).integers(-8, 9, shape).astype(np.float32)


def coded(lib, x, nseg=0, seed=0):
    """An FP8 tensor with these values as codes, under scales that are powers of two."""
    q = lib.FP8.empty(*x.shape, nseg)
    q.codes.copy_(torch.from_numpy(M.encode(x)))
    q.scales.copy_(torch.from_numpy(np.exp2(synth.rng(seed).integers(-1, 2, q.scales.shape)).astype(np.float32)))
    return q


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("K,N,epi", [(16, 8, 0), (400, 288, 0), (1040, 33, 0), (528, 288, 1), (384, 768, 1)])
def test_exact_sums_are_the_same_in_every_type(gpu_lib, counts, K, N, epi):
    """Sums of integers: the BF16 rows are the FP32 rows rounded, whichever instruction makes them."""
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    a = coded(gpu_lib, small_integers((R, K), 1), seed=2)
    b = coded(gpu_lib, small_integers((E * N * (1 + epi), K), 3), E, 4)
    o = dict(M_cap=R, epilogue=epi)
    C = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, **o)
    if not epi:
        assert np.array_equal(host(C), moe.grouped_gemm_m(vals(a), tile_vals(b), off, E, N))
    C16 = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, out_dtype=torch.bfloat16, **o)
    assert same_bits(C16, C.bfloat16())
    if epi:
        for ct in (torch.float32, torch.bfloat16, None):
            q = gpu_lib.FP8.empty(R, N)
            got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, q_out=q, want_c=ct is not None,
                                           out_dtype=ct or torch.float32, **o)
            check_codes(q, host(C))
            assert got is None if ct is None else same_bits(got, C.to(ct))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("counts,N", [([130, 0, 77, 300], 32), ([130, 0, 77, 300], 96), ([1, 0, 3, 2], 224),
                                      ([500, 900, 0, 77], 768), ([3, 1, 0, 0], 768)])
def test_swiglu_requantised_in_the_epilogue(gpu_lib, counts, N, rule):
    E, K, off = 4, 416, np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    aq = gpu_lib.fp8_quantize(dev_bf16(synth.activations(R, K, 1)))
    bq = weights(gpu_lib, E, 2 * N, K, 2)
    o = dict(M_cap=R, epilogue=gpu_lib.NV4_EPI_SWIGLU)
    plain = gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, **o)
    ref = check_product(host(plain), vals(aq), tile_vals(bq), off, E, N, swiglu=True)
    for ct in (torch.float32, torch.bfloat16):
        q = gpu_lib.FP8.empty(R + 1, N)
        q.codes.fill_(0xEE)
        q.scales.fill_(7.0)
        part = gpu_lib.FP8(q.codes[:R], q.scales[:R], R, N)
        C = torch.empty((R, N + 8), dtype=ct, device="cuda")[:, :N]
        gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, C=C, q_out=part, rule=rule, **o)
        if ct == torch.float32:
            # (small problems without q_out take another kernel, with another order of the sum over K)
            assert R < 1000 or same_bits(C.contiguous(), plain)
            check_product(host(C), vals(aq), tile_vals(bq), off, E, N, swiglu=True)
            check_codes(part, host(C.contiguous()), rule)
        else:
            assert R < 1000 or same_bits(C.contiguous(), gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, out_dtype=ct, **o))
            check_product(host(C), vals(aq), tile_vals(bq), off, E, N, swiglu=True, bf16=True)
            # the codes of a result that is itself between two BF16 values: half a BF16 step and half a code step
            v, c = vals(part), host(C).astype(np.float64)
            G = np.repeat(host(part.scales).astype(np.float64), 128, 1)[:, :N]
            assert (np.abs(v - c) <= HALF_BF16 * np.abs(c) + (2.0 ** -4 * np.abs(v) + 2.0 ** -10 * G) * (1 + 1e-6)).all()
            rel = np.linalg.norm(v - ref) / np.linalg.norm(ref)
            assert rel <= 2.0 ** -4 + CUT
        assert (q.codes[R] == 0xEE).all() and (q.scales[R] == 7.0).all()
    alone = gpu_lib.FP8.empty(R, N)
    assert gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, q_out=alone, want_c=False, rule=rule, **o) is None
    assert same_bits(alone.codes, part.codes) and same_bits(alone.scales, part.scales)


def test_gather_is_the_materialised_gather(gpu_lib):
    counts, K, N, E = [70, 0, 300, 9], 336, 96, 4
    off = np.concatenate([[0], np.cumsum(counts)])
    R, T = int(off[-1]), 100
    x = synth.activations(T, K, 7)
    idx = synth.rng(8).integers(0, T, R).astype(np.int32)
    aq, ag = gpu_lib.fp8_quantize(dev_bf16(x)), gpu_lib.fp8_quantize(dev_bf16(x[idx]))
    bq = weights(gpu_lib, E, N, K, 2)
    one = gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, a_rows=dev_i32(idx))
    two = gpu_lib.fp8_grouped_gemm(ag, bq, dev_i32(off), E, N, M_cap=R)
    assert same_bits(one, two)
    # rows outside A are clamped into it, and M_cap cuts the last rows off
    idx2 = idx.copy()
    idx2[:2] = [-9, T + 5]
    idx[:2] = [0, T - 1]
    out = torch.full((R, N), 7.0, device="cuda")
    gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R - 5, a_rows=dev_i32(idx2), C=out)
    ref = gpu_lib.fp8_grouped_gemm(aq, bq, dev_i32(off), E, N, M_cap=R, a_rows=dev_i32(idx))
    assert same_bits(out[:R - 5].contiguous(), ref[:R - 5].contiguous()) and (out[R - 5:] == 7.0).all()


def test_nan_block_reaches_its_results_only(gpu_lib):
    x = synth.activations(40, 256, 1)
    x[3, 5] = np.nan
    aq = gpu_lib.fp8_quantize(dev_bf16(x))
    w = synth.weights((192, 256), 2)
    off = dev_i32(np.array([0, 40]))
    C = host(gpu_lib.fp8_grouped_gemm(aq, gpu_lib.fp8_quantize(dev_bf16(w), layout=gpu_lib.NV4_F8_TILES), off, 1, 192))
    assert np.isnan(C[3]).all() and np.isfinite(np.delete(C, 3, 0)).all()
    w[150, 3] = np.inf                                          # the second block row of the weights
    C = host(gpu_lib.fp8_grouped_gemm(aq, gpu_lib.fp8_quantize(dev_bf16(w), layout=gpu_lib.NV4_F8_TILES), off, 1, 192))
    assert np.isnan(C[:, 128:]).all() and np.isfinite(np.delete(C, 3, 0)[:, :128]).all()


@pytest.mark.parametrize("counts", [[1], [0, 5, 0, 128], [300, 0, 129, 7, 0], [40, 1200, 3]])
@pytest.mark.parametrize("N,Mc", [(16, 16), (64, 288), (320, 96), (48, 130)])
@pytest.mark.parametrize("rules", [(M.FP32, M.FP32), (M.POW2, M.POW2), (M.FP32, M.POW2)])
def test_group_k(gpu_lib, counts, N, Mc, rules):
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    Mp = (Mc + 15) // 16 * 16
    a, b = synth.gradients((R, N), 4), synth.activations(R, Mp, 5)
    po = gpu_lib.mx_padded_offsets(dev_i32(off))
    cols = lambda t, rule: gpu_lib.fp8_quantize(dev_bf16(t), layout=gpu_lib.NV4_COLS, nseg=E, seg_offsets=dev_i32(off),
                                                seg_padded_offsets=po, rule=rule)
    aq, bq = cols(a, rules[0]), cols(b, rules[1])
    bq = gpu_lib.FP8(bq.codes[:Mc], bq.scales[:Mc], Mc, bq.K, rule=bq.rule)
    # NaN scales behind the last segment must not matter
    rpo = MX.padded_offsets(off)
    P = int(rpo[-1])
    aq.scales[:, P // 128:] = float("nan")
    C = gpu_lib.fp8_grouped_gemm(aq, bq, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K)
    av, bv = [M.values(host(q.codes)[:, :P], host(q.scales)[:, :P // 128]) for q in (aq, bq)]
    ref = moe.grouped_gemm_k(av, bv, rpo, E)
    pad = max(counts) + 128
    tol = moe.grouped_gemm_k(np.abs(av), np.abs(bv), rpo, E) * ULP * (pad + 3 * (pad // 128 + 1))
    assert (np.abs(host(C) - ref) <= tol).all()
    for e in range(E):
        if counts[e] == 0:
            assert (host(C)[e] == 0).all()
    C16 = gpu_lib.fp8_grouped_gemm(aq, bq, po, E, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=torch.bfloat16)
    tol += moe.grouped_gemm_k(np.abs(av), np.abs(bv), rpo, E) * CUT
    assert (np.abs(host(C16) - ref) <= tol + HALF_BF16 * (np.abs(ref) + tol)).all()


def test_group_k_exact_sums_and_whole_blocks(gpu_lib):
    """Integers: BF16 is FP32 rounded; ranges that are not whole blocks are taken to the blocks they touch."""
    a, b = coded(gpu_lib, small_integers((48, 512), 1), seed=2), coded(gpu_lib, small_integers((130, 512), 3), seed=4)
    k = dict(group_mode=gpu_lib.NV4_GROUP_K)
    off = dev_i32(np.array([0, 128, 128, 512]))
    C = gpu_lib.fp8_grouped_gemm(a, b, off, 3, 0, **k)
    assert np.array_equal(host(C), moe.grouped_gemm_k(vals(a), vals(b), [0, 128, 128, 512], 3))
    assert same_bits(gpu_lib.fp8_grouped_gemm(a, b, off, 3, 0, out_dtype=torch.bfloat16, **k), C.bfloat16())
    C = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(np.array([5, 100, 129, 900])), 3, 0, **k)
    for e, (lo, hi) in enumerate([(0, 128), (0, 256), (128, 512)]):
        assert np.array_equal(host(C)[e], vals(a)[:, lo:hi] @ vals(b)[:, lo:hi].T)


@pytest.mark.parametrize("N,ld,first", [(96, 96, 0), (96, 98, 1), (96, 97, 0), (95, 96, 0), (95, 95, 0), (352, 360, 3),
                                        (1, 1, 0), (2, 4, 2), (351, 352, 0), (352, 352, 0)])
@pytest.mark.parametrize("rows", [70, 900, 5000])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_results_of_any_alignment(gpu_lib, N, ld, first, rows, dt):
    """Every tile, column counts and row strides that do and do not allow wide stores: the same rows, and
    nothing else is written."""
    E, K = 2, 160
    off = dev_i32(np.array([0, rows // 3, rows - 2]))
    a = gpu_lib.fp8_quantize(torch.randn(rows, K, device="cuda"))
    for epi in (0, 1) if N % 32 == 0 else (0,):
        b = gpu_lib.fp8_quantize(torch.randn(E * N * (1 + epi), K, device="cuda"), layout=gpu_lib.NV4_F8_TILES, nseg=E)
        ref = gpu_lib.fp8_grouped_gemm(a, b, off, E, N, M_cap=rows, epilogue=epi, out_dtype=dt)
        big = torch.full((rows * ld + first + 64,), 3.0, dtype=dt, device="cuda")
        C = big[first:first + rows * ld].view(rows, ld)[:, :N]
        gpu_lib.fp8_grouped_gemm(a, b, off, E, N, M_cap=rows, epilogue=epi, C=C)
        assert same_bits(C[:rows - 2].contiguous(), ref[:rows - 2].contiguous())
        C[:rows - 2] = 3.0
        assert (big == 3.0).all()


def test_empty_calls(gpu_lib):
    q = gpu_lib.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert q.rows == 0 and gpu_lib.fp8_dequantize(q).shape == (0, 64)
    w = weights(gpu_lib, 2, 32, 64, 1)
    assert gpu_lib.fp8_grouped_gemm(q, w, dev_i32(np.zeros(3)), 2, 32).shape == (0, 32)
    a = gpu_lib.fp8_quantize(torch.randn(5, 64, device="cuda"))
    C = torch.full((5, 32), 9.0, device="cuda")
    gpu_lib.fp8_grouped_gemm(a, w, dev_i32(np.zeros(3)), 2, 32, C=C)
    assert (C == 9.0).all()
