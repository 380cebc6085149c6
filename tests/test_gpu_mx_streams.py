"""MXFP4 calls on a stream of their own while the current one is busy: where their memory comes
from, and that neither stream's results change."""

import pytest
import torch

from tests.gpu_util import same_bits
from tests.test_gpu_mx import dev_bf16, dev_f32, few_case

pytestmark = pytest.mark.gpu


def pool_of(t):
    """The stream whose pool holds t's memory."""
    p = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= p < s["address"] + s["total_size"])


def keep_busy(n=20):
    """Some milliseconds of work for the current stream, so that what is queued behind it is still
    pending when the host goes on."""
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda")
    for _ in range(n):
        torch.mm(a, a)


def test_outputs_come_from_the_streams_pool(gpu_lib):
    T, E, k, H, I = 12, 16, 4, 256, 64
    x, lg, w, *_ = few_case(gpu_lib, T, E, k, H, I)
    x, lg, s = dev_bf16(x), dev_f32(lg), torch.cuda.Stream()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    q = gpu_lib.mxfp4_quantize(x, stream=s)
    outs = [q.codes, q.scales, gpu_lib.mxfp4_dequantize(q, stream=s), gpu_lib.mx_padded_offsets(off, stream=s),
            gpu_lib.mxfp4_grouped_gemm(q, w.w13, off, 1, E * 2 * I, stream=s),
            gpu_lib.mx_moe_few(x, lg, w, k, stream=s)]
    assert [pool_of(t) for t in outs] == [s.cuda_stream] * len(outs)
    assert pool_of(x) != s.cuda_stream
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 7, 40])
def test_a_call_behind_a_busy_stream_and_one_beside_it(gpu_lib, T):
    """Without ws: the first call's workspace is free for the current stream again when the call
    returns, with its kernels still pending.  The second must not get it."""
    E, k, H, I = 16, 4, 1024, 256
    x, lg, w, *_ = few_case(gpu_lib, 2 * T, E, k, H, I)
    x, lg = dev_bf16(x), dev_f32(lg)
    a, b = (x[:T], lg[:T]), (x[T:], lg[T:])
    want = gpu_lib.mx_moe_few(*a, w, k), gpu_lib.mx_moe_few(*b, w, k)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        keep_busy()
        outs.append((gpu_lib.mx_moe_few(*a, w, k), want[0]))
        for _ in range(3):
            outs.append((gpu_lib.mx_moe_few(*b, w, k, stream=s), want[1]))
        outs.append((gpu_lib.mx_moe_few(*a, w, k), want[0]))
    torch.cuda.synchronize()
    for got, ref in outs:
        assert same_bits(got, ref)


def layer_case(gpu_lib, T=96, E=8, k=2, H=256, I=64):
    x, lg, w, v13, v2 = few_case(gpu_lib, T, E, k, H, I)
    g = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, dtype=torch.bfloat16, device="cuda", generator=g)
    W13, W2 = rand(E, 2 * I, H), rand(E, H, I)
    return (dev_bf16(x), dev_f32(lg), w, gpu_lib.mx_quantize_expert_weights_t(W13, W2), rand(T * k, H),
            rand(T * k, 2 * I), (T, H, E, k, I))


def test_a_layer_on_a_stream_beside_a_busy_one(gpu_lib):
    """Without buffers of the caller's, each result taken from buffers that are dropped at once,
    forward and backward in turn on two streams."""
    x, lg, w, wt, dY2, dY13, shape = layer_case(gpu_lib)
    k = shape[3]
    results = lambda g: [g.dhact, g.dxperm, g.dw2, g.dw13]

    def step(**o):
        out = gpu_lib.mx_moe_forward(x, lg, w, k, **o).out
        # (the buffers are made on the stream that fills them)
        with torch.cuda.stream(o.get("stream")):
            f = gpu_lib.mx_alloc_forward(*shape, keep_hact=True)
        gpu_lib.mx_moe_forward(x, lg, w, k, f, **o)
        return [out] + results(gpu_lib.mx_moe_backward(x, f, wt, dY2, dY13, **o))

    want = step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        keep_busy()
        got += [step(), step(stream=s), step(stream=s), step()]
    f = gpu_lib.mx_moe_forward(x, lg, w, k, stream=s)
    assert [pool_of(t) for t in (f.out, f.y, f.pws, f.xq.codes, f.hq.scales, f.routing.offsets)] == [s.cuda_stream] * 6
    torch.cuda.synchronize()
    for ts in got:
        assert all(same_bits(a, b) for a, b in zip(ts, want))


def test_strided_weights_on_a_stream(gpu_lib):
    """The copy of weights whose rows are not in one stride, before and behind work of its size."""
    E, H, I = 6, 512, 256
    g = torch.Generator("cuda").manual_seed(2)
    W13 = torch.randn(2 * I, E, H, dtype=torch.bfloat16, device="cuda", generator=g).transpose(0, 1)
    W2 = torch.randn(H, E, I, dtype=torch.bfloat16, device="cuda", generator=g).transpose(0, 1)
    flat = lambda w, wt: [t for m in (w.w13, w.w2, wt.w13t, wt.w2t) for t in (m.codes, m.scales)]
    both = lambda a, b, **o: flat(gpu_lib.mx_quantize_expert_weights(a, b, **o),
                                  gpu_lib.mx_quantize_expert_weights_t(a, b, **o))
    want = both(W13.contiguous(), W2.contiguous())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        keep_busy()
        got += [both(W13, W2, stream=s), both(W13, W2)]
    torch.cuda.synchronize()
    for ts in got:
        assert all(same_bits(a, b) for a, b in zip(ts, want))
    assert pool_of(got[0][0]) == s.cuda_stream


def test_captured_on_a_forked_stream(gpu_lib):
    """Calls with `stream` of a stream forked into a capture: their memory belongs to the graph, whose
    replays between eager calls on either stream give the eager results."""
    T, E, k, H, I = 20, 16, 4, 256, 64
    x, lg, w, *_ = few_case(gpu_lib, 2 * T, E, k, H, I)
    xs, ls = dev_bf16(x), dev_f32(lg)
    x, lg = xs[:T].clone(), ls[:T].clone()
    s = torch.cuda.Stream()

    def step(o):
        few = gpu_lib.mx_moe_few(x, lg, w, k, **o)
        f = gpu_lib.mx_moe_forward(x, lg, w, k, **o)
        return [few, f.out, gpu_lib.mxfp4_dequantize(gpu_lib.mxfp4_quantize(x, **o), **o)]

    step({})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        got = step(dict(stream=s))
        here.wait_stream(s)
    for i in range(4):
        x.copy_(xs[i * 5:i * 5 + T])
        lg.copy_(ls[i * 5:i * 5 + T])
        want = step({})
        torch.cuda.synchronize()
        beside = step(dict(stream=s))
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, beside):
            assert same_bits(a, b) and same_bits(c, b)
