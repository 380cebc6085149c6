"""The MXFP4 layer with its options: renormalised weights, the ceiling rule, BF16 expert rows, FP32
tokens and strided ones, one token, all experts chosen."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from oracle import mxfp4 as M
from tests.gpu_util import bf16_rne_of, dev_bf16, dev_f32, host, rel_frob, same_bits
from tests.test_gpu_mx import check_codes, check_product, vals

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,H,I", [(1, 3, 3, 64, 32), (77, 5, 5, 96, 160), (300, 40, 6, 160, 64)])
@pytest.mark.parametrize("rule", [M.FLOOR, M.CEIL])
@pytest.mark.parametrize("y_dtype", [torch.float32, torch.bfloat16])
def test_forward(gpu_lib, T, E, k, H, I, rule, y_dtype):
    x, lg = synth.activations(T, H, 1), synth.logits_softmax(T, E, 2)
    W13, W2 = synth.weights((E, 2 * I, H), 3), synth.weights((E, H, I), 4)
    w = gpu_lib.mx_quantize_expert_weights(dev_bf16(W13), dev_f32(W2), rule=rule)
    check_codes(w.w13, W13.reshape(-1, H), rule)
    check_codes(w.w2, W2.reshape(-1, I), rule)
    wide = torch.full((T, H + 16), 3.0, device="cuda")
    wide[:, 8:8 + H] = dev_f32(x)
    f = gpu_lib.mx_alloc_forward(T, H, E, k, I, out_dtype=torch.float32, y_dtype=y_dtype, rule=rule)
    gpu_lib.mx_moe_forward(wide[:, 8:8 + H], dev_f32(lg), w, k, f, flags=gpu_lib.NV4_RENORM)
    ids, wts = moe.route_topk(lg, k, renorm=True)
    p = moe.permute(ids, E)
    off, rt = p["offsets"], p["row_token"]
    assert np.array_equal(host(f.routing.topk_ids), ids) and rel_frob(host(f.routing.topk_w), wts) <= 1e-6
    check_codes(f.xq, x, rule)
    o = f.routing.offsets
    h = gpu_lib.mxfp4_grouped_gemm(f.xq, w.w13, o, E, I, M_cap=T * k, a_rows=f.routing.row_token,
                                   epilogue=gpu_lib.NV4_EPI_SWIGLU)
    check_product(host(h), vals(f.xq)[rt], vals(w.w13), off, E, I, swiglu=True)
    check_codes(f.hq, host(h), rule)
    y = gpu_lib.mxfp4_grouped_gemm(f.hq, w.w2, o, E, H)
    check_product(host(y), vals(f.hq), vals(w.w2), off, E, H)
    assert np.array_equal(host(f.y), host(y) if y_dtype == torch.float32 else bf16_rne_of(host(y)))
    assert rel_frob(host(f.out), moe.combine(host(f.y), p["token_row"], host(f.routing.topk_w).astype(np.float64))) <= 1e-5
    # the same buffers again, from BF16 tokens (their values are BF16's)
    first = f.out.clone()
    f.out.zero_()
    gpu_lib.mx_moe_forward(dev_bf16(x), dev_f32(lg), w, k, f, flags=gpu_lib.NV4_RENORM)
    assert same_bits(f.out, first)
