"""Uneven loads: the MXFP4 products' tiles and the few-token layer's ways are chosen by the mean rows
of an expert, and have to be right when one expert has them all."""

import numpy as np
import pytest
import torch

import synth
from tests.gpu_util import bf16_rne_of, dev_bf16, dev_f32, dev_i32, host
from tests.test_gpu_mx import check_codes, check_product, few_case, few_reference, vals

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,chosen", [
    (64, 256, 2, 2), (64, 1024, 2, 3), (63, 128, 1, 1), (16, 300, 8, 9),   # by assignments
    (64, 16, 8, 8), (33, 64, 4, 4), (64, 200, 8, 10)])                     # grouped
def test_few_tokens_of_few_experts(gpu_lib, T, E, k, chosen):
    """Every token takes k of the same `chosen` experts."""
    H, I = 160, 96
    x, _, w, v13, v2 = few_case(gpu_lib, T, E, k, H, I, seed=T)
    r = synth.rng(E)
    mine = r.choice(E, chosen, replace=False)
    ids = np.stack([r.permutation(mine)[:k] for _ in range(T)]).astype(np.int32)
    wts = (r.random((T, k)) + 0.1).astype(np.float32)
    routed = dict(topk_ids=dev_i32(ids), topk_w=dev_f32(wts))
    out = gpu_lib.mx_moe_few(dev_bf16(x), None, w, k, out_dtype=torch.float32, **routed)
    ref, tol = few_reference(x, ids, wts.astype(np.float64), v13, v2)
    assert (np.abs(host(out) - ref) <= tol + 1e-38).all()
    again = gpu_lib.mx_moe_few(dev_bf16(x), None, w, k, **routed)
    assert np.array_equal(host(again), bf16_rne_of(host(out)))


@pytest.mark.parametrize("hot", [0, 70, 127])
@pytest.mark.parametrize("epi", [0, 1])
def test_a_hot_expert_in_the_smallest_tile(gpu_lib, hot, epi):
    """128 experts with less than 64 rows each in the mean, of which one has five sixths."""
    E, K, N = 128, 416, 96
    counts = synth.rng(hot).integers(0, 12, E)
    counts[hot] = 4000
    off = np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    assert R < 64 * E
    aq = gpu_lib.mxfp4_quantize(dev_bf16(synth.activations(R, K, 1)))
    bq = gpu_lib.mxfp4_quantize(dev_bf16(synth.weights((E * N * (1 + epi), K), 2)))
    C = gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, epilogue=epi)
    check_product(host(C), vals(aq), vals(bq), off, E, N, swiglu=bool(epi))
    if epi:
        q = gpu_lib.MXFP4.empty(R, N)
        gpu_lib.mxfp4_grouped_gemm(aq, bq, dev_i32(off), E, N, epilogue=epi, q_out=q, want_c=False)
        check_codes(q, host(C))
