"""The FP8 product with weights above 4 GiB, bit for bit and by every kernel, and the FP8 layer at a prompt's size."""

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as M
from tests.gpu_util import dev_bf16, dev_f32, dev_i32, same_bits
from tests.test_gpu_f8 import CUT, HALF_BF16, ULP
from tests.test_gpu_f8_tiles import BF16, F32, coded, reference, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far_weights():
    """132 experts of 8192 x 4096, NaN but for the first and the last; and those two alone."""
    import nvfp4_w4a4_moe_amd as lib
    E, N, K = 132, 8192, 4096
    two = coded(lib, 2 * N, K, 2, 2, M.POW2)
    w = lib.FP8.empty(E * N, K, E)
    w.codes.fill_(0x7F)
    w.scales.fill_(float("nan"))
    for e, src in ((0, 0), (E - 1, 1)):
        w.codes[e * N:(e + 1) * N] = two.codes[src * N:(src + 1) * N]
        w.scales[e] = two.scales[src]
    assert w.codes.numel() > 1 << 32
    return w, two, E, N, K


# rows that the kernel for few, and the tiles of 64, 128 and 256 rows take
@pytest.mark.parametrize("R", [2, 700, 9000, 20000])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_weights_above_4_gib(gpu_lib, far_weights, R, rule, dt):
    w, two, E, N, K = far_weights
    w.rule = rule
    a = coded(gpu_lib, R, K, 0, 3, rule)
    off = np.array([0] + [R // 2] * (E - 1) + [R])
    ref = reference(a, two, [0, R // 2, R], 2, N)
    assert same_bits(gpu_lib.fp8_grouped_gemm(a, w, dev_i32(off), E, N, out_dtype=dt), ref.to(dt))
    a.scales.mul_(2.0 ** -10)
    o = dict(M_cap=R, epilogue=gpu_lib.NV4_EPI_SWIGLU, out_dtype=dt)
    got = gpu_lib.fp8_grouped_gemm(a, w, dev_i32(off), E, N // 2, **o)
    near = gpu_lib.FP8(two.codes, two.scales, 2 * N, K, 2, rule)
    assert same_bits(got, gpu_lib.fp8_grouped_gemm(a, near, dev_i32(np.array([0, R // 2, R])), 2, N // 2, **o))
    assert got.isfinite().all()


def tiles64(q):
    """FP64 values [nseg, m, K] of a tensor in 128 x 128 blocks."""
    return values(q).double().view(q.nseg, -1, q.K)


@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_layer_of_a_prompt(gpu_lib, rule):
    """4096 tokens, 8 experts, two each: stage by stage on the layer's own operands, in 64 bits."""
    T, E, k, H, I = 4096, 8, 2, 1024, 768
    x, lg = dev_bf16(synth.activations(T, H, 1)), dev_f32(synth.logits_softmax(T, E, 2))
    w = gpu_lib.fp8_quantize_expert_weights(dev_bf16(synth.weights((E, 2 * I, H), 3)), dev_bf16(synth.weights((E, H, I), 4)),
                                            rule=rule)
    f = gpu_lib.fp8_alloc_forward(T, H, E, k, I, keep_hact=True, out_dtype=F32, rule=rule)
    gpu_lib.fp8_moe_forward(x, lg, w, k, f)
    rt = f.routing
    off, rows = rt.offsets.tolist(), rt.row_token.long()
    want = gpu_lib.fp8_quantize(x, rule=rule)
    assert same_bits(f.xq.codes, want.codes) and same_bits(f.xq.scales, want.scales)
    a, w13 = values(f.xq).double()[rows], tiles64(w.w13)
    h, tol = torch.empty(T * k, I, dtype=torch.float64, device="cuda"), torch.empty(T * k, I, dtype=torch.float64, device="cuda")
    # The sums' error: K roundings and scalings of FP32, and the matrix instruction's cut.  Through SwiGLU: silu's slope is at
    # most 1.1 and |silu(g)| <= |g|; its own error (1.25 |g| + 8) 2^-24.
    per = ULP * (H + 3 * (H // 128)) + CUT
    for e in range(E):
        s = slice(off[e], off[e + 1])
        y, m = a[s] @ w13[e].T, a[s].abs() @ w13[e].abs().T * per
        g, u, mg, mu = y[:, :I], y[:, I:], m[:, :I], m[:, I:]
        h[s] = g * torch.sigmoid(g) * u
        tol[s] = 1.1 * mg * (u.abs() + mu) + g.abs() * mu + h[s].abs() * (1.25 * g.abs() + 8) * 2.0 ** -24
    assert ((f.hact.double() - h).abs() <= tol + HALF_BF16 * (h.abs() + tol)).all()
    # codes of the unrounded result: half a code step (e4m3: 2^-4 of the value, 2^-10 of the scale below the normal ones)
    hv, G = values(f.hq).double(), f.hq.scales.double().repeat_interleave(128, 1)[:, :I]
    assert ((hv - h).abs() <= tol + (2.0 ** -4 * hv.abs() + 2.0 ** -10 * G) * (1 + 1e-6)).all()
    w2 = tiles64(w.w2)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        y, m = hv[s] @ w2[e].T, hv[s].abs() @ w2[e].abs().T
        assert ((f.y[s].double() - y).abs() <= m * ULP * (I + 3 * (I // 128))).all()
    mixed = (f.y.double()[rt.token_row.long()] * rt.topk_w.double()[..., None])
    assert ((f.out.double() - mixed.sum(1)).abs() <= k * 2.0 ** -23 * mixed.abs().sum(1)).all()
