"""The FP8 and router binding on the CPU: what it passes to the library, on which stream, and what it
refuses (with the stand-in library and tensors of the MXFP4 binding's tests)."""

import pytest
import torch

import nvfp4_w4a4_moe_amd as nv4
from nvfp4_w4a4_moe_amd import fp8, router
from tests.test_mx_binding import BF16, OVERLAPPING, Gpu, Stream, i32, layer_tensors, ten

F32 = torch.float32


@pytest.fixture
def gpu(monkeypatch):
    g = Gpu(monkeypatch)
    for module in (fp8, router):
        monkeypatch.setattr(module, "load", lambda: g)
    yield g
    Gpu.now = None


def f8(rows, K, nseg=0):
    shape = (nseg, -(-(rows // nseg) // 128), -(-K // 128)) if nseg else (rows, -(-K // 128))
    return nv4.FP8(ten(rows, K, dtype=torch.uint8), ten(*shape, dtype=F32), rows, K, nseg)


def weights(E, H, I):
    return nv4.F8ExpertWeights(f8(E * 2 * I, H, E), f8(E * H, I, E), E, H, I)


def balance(nseg, E):
    return nv4.MoeBalance(ten(2, dtype=F32), ten(nseg, E, dtype=torch.int32), ten(nseg, E, dtype=F32),
                          ten(nseg, dtype=torch.int32))


# ----------------------------------------------------------------------------- strides

@pytest.mark.parametrize("make", OVERLAPPING)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_overlap_are_refused(gpu, make, dtype):
    bad = make(3, dtype)
    for call in (lambda: nv4.fp8_quantize(bad), lambda: nv4.fp8_quantize(bad, row_index=i32(0, 1, 2, 2)),
                 lambda: nv4.fp8_quantize(bad, layout=nv4.NV4_F8_TILES), lambda: nv4.fp8_dequantize(f8(3, 64), out=bad),
                 lambda: nv4.fp8_grouped_gemm(f8(3, 96), f8(64, 96, 1), i32(0, 3), 1, 64, C=bad),
                 lambda: nv4.moe_combine_backward(ten(3, 64), bad, i32(0, 1, 2).view(3, 1), ten(3, 1, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(3, 64), ten(3, 64, dtype=dtype), i32(0, 1, 2).view(3, 1),
                                                  ten(3, 1, dtype=F32), dY=bad)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert not gpu.calls


def test_row_strides_are_the_tensors(gpu):
    wide = ten(5, 96)
    for x, ldx in ((wide, 96), (wide[:, :64], 96), (wide[::2, 32:], 192), (wide[:1, :64], 64), (ten(64).expand(1, 64), 64)):
        nv4.fp8_quantize(x)
        assert gpu.args("fp8_quantize")[-1][5] == ldx
        nv4.fp8_dequantize(f8(*x.shape), out=x)
        assert gpu.args("fp8_dequantize")[-1][3] == ldx
        nv4.fp8_grouped_gemm(f8(x.shape[0], 96), f8(x.shape[1], 96, 1), i32(0, 1), 1, x.shape[1], C=x)
        assert gpu.args("fp8_grouped_gemm")[-1][11] == ldx
        n = x.shape[0]
        nv4.moe_combine_backward(ten(n, x.shape[1]), x, i32(*range(n)).view(n, 1), ten(n, 1, dtype=F32))
        a = gpu.args("moe_combine_backward")[-1]
        assert a[4] == ldx and a[5] == n and a[12] == x.shape[1]


def test_descriptors(gpu):
    """Shapes, grouping and rule of every operand as the library sees them."""
    d = lambda t: (t.rows, t.K, t.nseg, t.rule)
    q = nv4.fp8_quantize(ten(300, 80), rule=nv4.NV4_F8_POW2)
    assert q.scales.shape == (300, 1) and d(q) == (300, 80, 0, 1)
    q = nv4.fp8_quantize(ten(600, 144), layout=nv4.NV4_F8_TILES, nseg=2)
    assert q.scales.shape == (2, 3, 2) and d(gpu.args("fp8_quantize")[-1][12]) == (600, 144, 2, 0) and q.nseg == 2
    q.rule = nv4.NV4_F8_POW2
    t = nv4.fp8_transpose(q) if q.rows // 2 % 16 == 0 else nv4.fp8_transpose(f8(64, 144, 2))
    assert t.scales.shape == (2, 2, 1) and d(gpu.args("fp8_transpose")[-1][1])[:3] == (288, 32, 2)
    seg = dict(nseg=2, seg_offsets=i32(0, 5, 9), seg_padded_offsets=i32(0, 128, 256))
    q = nv4.fp8_quantize(ten(9, 32), layout=nv4.NV4_ROWS_AND_COLS, rule=nv4.NV4_F8_POW2, **seg)
    assert d(q) == (32, nv4.mx_cols_capacity(9, 2), 0, 1) and d(q.rows_out) == (9, 32, 0, 1)
    # a buffer of another grouping is taken if its scales fit, and described anew
    out = f8(128, 128, 1)
    out.scales = ten(128, 1, dtype=F32)
    assert d(nv4.fp8_quantize(ten(128, 128), out=out)) == (128, 128, 0, 0)
    with pytest.raises(ValueError, match="nseg 1"):
        nv4.fp8_quantize(ten(128, 128), layout=nv4.NV4_F8_TILES, out=out)
    with pytest.raises(ValueError, match="equal matrices"):
        nv4.fp8_quantize(ten(5, 64), layout=nv4.NV4_F8_TILES, nseg=2)
    with pytest.raises(ValueError, match="128 x 128"):
        nv4.fp8_transpose(f8(64, 64))


@pytest.mark.parametrize("shape", [(2, 9, 64), (2, 7, 64), (2, 8, 65), (3, 8, 64), (16, 64)])
def test_weight_gradients_have_their_own_shape(gpu, shape):
    o = dict(group_mode=nv4.NV4_GROUP_K)
    a, b, off = f8(8, 128), f8(64, 128), i32(0, 128, 128)
    with pytest.raises(ValueError, match=r"C must be \[2, 8, 64\]"):
        nv4.fp8_grouped_gemm(a, b, off, 2, 0, C=ten(*shape), **o)
    assert not gpu.calls
    assert nv4.fp8_grouped_gemm(a, b, off, 2, 0, C=ten(2, 8, 64), **o).shape == (2, 8, 64)
    assert gpu.args("fp8_grouped_gemm")[-1][11] == 64


# ----------------------------------------------------------------------------- devices

def test_tensors_on_another_device_are_refused(gpu):
    far = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype)
    half = lambda rows, K, nseg=0: nv4.FP8(f8(rows, K, nseg).codes, far(*f8(rows, K, nseg).scales.shape), rows, K, nseg)
    x, seg = ten(4, 64), dict(nseg=1, seg_offsets=i32(0, 4), seg_padded_offsets=i32(0, 128))
    lg, ids, row = ten(4, 8, dtype=F32), i32(*range(8)).view(4, 2), i32(*range(8)).view(4, 2)
    b, dl = balance(1, 8), ten(2, dtype=F32)
    farb = nv4.MoeBalance(b.loss, far(1, 8, dtype=torch.int32), b.prob_sums, b.tokens)
    w = ten(4, 2, dtype=F32)
    for call in (lambda: nv4.fp8_quantize(x, out=half(4, 64)),
                 lambda: nv4.fp8_quantize(x, layout=nv4.NV4_ROWS_AND_COLS, out=f8(64, 256), out_rows=half(4, 64), **seg),
                 lambda: nv4.fp8_dequantize(half(4, 64)), lambda: nv4.fp8_transpose(half(32, 64, 2)),
                 lambda: nv4.fp8_transpose(f8(32, 64, 2), out=half(128, 16, 2)),
                 lambda: nv4.fp8_grouped_gemm(f8(4, 64), half(64, 64, 1), i32(0, 4), 1, 64),
                 lambda: nv4.fp8_grouped_gemm(f8(4, 64), f8(64, 64, 1), i32(0, 4), 1, 32, epilogue=nv4.NV4_EPI_SWIGLU,
                                              q_out=half(4, 32), want_c=False),
                 lambda: nv4.moe_balance_loss(lg, far(4, 2, dtype=torch.int32)),
                 lambda: nv4.moe_balance_loss(lg, ids, mask=far(4, dtype=torch.bool)),
                 lambda: nv4.moe_balance_loss(lg, ids, out=farb),
                 lambda: nv4.moe_balance_backward(lg, ids, farb, dl),
                 lambda: nv4.moe_balance_backward(lg, ids, b, far(2)),
                 lambda: nv4.moe_balance_backward(lg, ids, dtopk_w=far(4, 2)),
                 lambda: nv4.moe_combine_backward(x, far(8, 64, dtype=BF16), row, w),
                 lambda: nv4.moe_combine_backward(x, ten(8, 64), row, far(4, 2))):
        with pytest.raises(ValueError, match="tensors on"):
            call()
    assert not gpu.calls


# ----------------------------------------------------------------------------- streams

def single_calls(stream):
    """Each call that makes its own outputs or workspace, as (call, its tensors)."""
    x, off, lg = ten(3, 64), i32(0, 3), ten(3, 4, dtype=F32)
    o = dict(stream=stream)
    both = dict(layout=nv4.NV4_ROWS_AND_COLS, seg_offsets=off, seg_padded_offsets=i32(0, 128))
    pair = lambda q: [q.codes, q.scales]
    ids, row, w = i32(*range(6)).view(3, 2), i32(*range(6)).view(3, 2), ten(3, 2, dtype=F32)
    return [lambda: pair(nv4.fp8_quantize(x, **o)),
            lambda: pair(nv4.fp8_quantize(x, layout=nv4.NV4_F8_TILES, **o)),
            lambda: sum(map(pair, (lambda q: (q, q.rows_out))(nv4.fp8_quantize(x, **both, **o))), []),
            lambda: [nv4.fp8_dequantize(f8(3, 64), **o)], lambda: pair(nv4.fp8_transpose(f8(32, 64, 2), **o)),
            lambda: [nv4.fp8_grouped_gemm(f8(3, 64), f8(32, 64, 1), off, 1, 32, **o)],
            lambda: list(vars(nv4.moe_balance_loss(lg, ids, **o)).values()),
            lambda: [nv4.moe_balance_backward(lg, ids, balance(1, 4), ten(2, dtype=F32), **o)],
            lambda: list(nv4.moe_combine_backward(x, ten(6, 64), row, w, **o))]


@pytest.mark.parametrize("i", range(9))
def test_a_streams_call_takes_the_streams_memory(gpu, i):
    call = single_calls(Stream(200))[i]
    gpu.made.clear()
    outs = call()
    assert gpu.calls and {s for *_, s, _ in gpu.calls} == {200}
    assert gpu.made and set(gpu.made.values()) == {200}
    assert {t.data_ptr() for t in outs} == {a for a, s in gpu.recorded.items() if s == {100}} == set(gpu.recorded)
    assert gpu.stream == Stream(100)


@pytest.mark.parametrize("i", range(9))
@pytest.mark.parametrize("given", [None, 100])
def test_the_current_streams_call_stays_there(gpu, i, given):
    call = single_calls(given and Stream(given))[i]
    gpu.made.clear()
    call()
    assert {s for *_, s, _ in gpu.calls} == {100} == set(gpu.made.values()) and not gpu.recorded


T, E, K_, H, I = 3, 4, 2, 64, 32


def forward(stream=None, bufs=None, n=T):
    return nv4.fp8_moe_forward(ten(n, H), ten(n, E, dtype=F32), weights(E, H, I), K_, bufs, stream=stream)


def backward(fwd, stream=None, bufs=None, dy2=(T * K_, H), dy13=(T * K_, 2 * I), n=T):
    wt = nv4.F8TransposedWeights(f8(E * I, H, E), f8(E * H, 2 * I, E))
    return nv4.fp8_moe_backward(ten(n, H), fwd, wt, ten(*dy2), ten(*dy13), bufs, stream=stream)


LAYER_CALLS = {"fp8_quantize", "moe_permute", "fp8_grouped_gemm", "moe_combine", "mx_padded_offsets"}


@pytest.mark.parametrize("given", [None, 100, 200])
def test_a_layer_on_a_stream_takes_the_streams_memory(gpu, given):
    at = given or 100
    stream = given and Stream(given)
    kept = nv4.fp8_alloc_forward(T, H, E, K_, I, keep_hact=True)
    gpu.made.clear()
    f = forward(stream)
    assert {n for n, *_ in gpu.calls} == LAYER_CALLS - {"mx_padded_offsets"} and {s for *_, s, _ in gpu.calls} == {at}
    mine = {t.data_ptr() for t in layer_tensors(f)}
    assert mine <= set(gpu.made) and set(gpu.made.values()) == {at}
    assert gpu.recorded == ({a: {100} for a in mine} if at == 200 else {})
    gpu.made.clear(), gpu.recorded.clear()
    f = forward(stream, kept)
    gpu.made.clear(), gpu.recorded.clear(), gpu.calls.clear()
    forward(stream, kept)   # routing and all: nothing is made
    assert not gpu.made and not gpu.recorded and {s for *_, s, _ in gpu.calls} == {at}
    gpu.calls.clear()
    g = backward(f, stream)
    assert {s for *_, s, _ in gpu.calls} == {at} == set(gpu.made.values())
    assert gpu.recorded == ({t.data_ptr(): {100} for t in layer_tensors(g)} if at == 200 else {})
    gpu.made.clear(), gpu.recorded.clear()
    q = nv4.fp8_quantize_expert_weights(ten(2 * I, E, H).transpose(0, 1), ten(E, H, I), stream=stream)
    t = nv4.fp8_transpose_expert_weights(q, stream=stream)
    kept = {x.data_ptr() for m in (q.w13, q.w2, t.w13t, t.w2t) for x in (m.codes, m.scales)}
    assert kept <= set(gpu.made) and set(gpu.made.values()) == {at}
    assert set(gpu.recorded) == (kept if at == 200 else set())
    assert gpu.stream == Stream(100)
    for call in (lambda s: forward(s), lambda s: backward(f, s)):
        with pytest.raises(ValueError, match="stream of cuda:1"):
            call(Stream(200, "cuda:1"))


def test_a_layer_on_another_device_than_the_current_one(gpu):
    gpu.device = 1
    f = forward()
    backward(forward(None, nv4.fp8_alloc_forward(T, H, E, K_, I, keep_hact=True)))
    nv4.fp8_transpose_expert_weights(nv4.fp8_quantize_expert_weights(ten(E, 2 * I, H), ten(E, H, I)))
    forward(Stream(200), f)
    assert LAYER_CALLS | {"fp8_transpose"} == {n for n, *_ in gpu.calls}
    assert {d for *_, d in gpu.calls} == {0} and {s for *_, s, _ in gpu.calls} == {100, 200}
    assert gpu.device == 1


# ----------------------------------------------------------------------------- shapes

def test_a_layers_inputs_fit_together(gpu):
    fwd = lambda n=T, lg=(T, E), k=K_, h=H, bufs=None: nv4.fp8_moe_forward(ten(n, h), ten(*lg, dtype=F32), weights(E, H, I),
                                                                           k, bufs)
    for lg in ((T + 1, E), (T - 1, E), (T, E + 1), (T * E,)):
        with pytest.raises(ValueError, match="logits"):
            fwd(lg=lg)
    with pytest.raises(ValueError, match="columns"):
        fwd(h=96)
    alloc = lambda n=T, h=H, k=K_: nv4.fp8_alloc_forward(n, h, E, k, I, keep_hact=True)
    for other in (alloc(n=T + 1), alloc(k=1), alloc(k=3), alloc(h=96)):
        with pytest.raises(ValueError, match="bufs"):
            fwd(bufs=other)
    used = fwd(bufs=alloc())
    gpu.calls.clear()
    for o in (dict(n=T - 1), dict(n=2 * T), dict(dy2=(T * K_, I)), dict(dy2=(T, H)), dict(dy13=(T * K_, I))):
        with pytest.raises(ValueError, match="rows|dY2"):
            backward(used, **o)
    with pytest.raises(ValueError, match="keep_hact"):
        backward(forward())
    gpu.calls.clear()
    for s13, s2 in (((E, 2 * I, H), (E, I, H)), ((E, 2 * I + 1, H), (E, H, I)), ((E, 2 * I, H), (E + 1, H, I))):
        with pytest.raises(ValueError, match="W2"):
            nv4.fp8_quantize_expert_weights(ten(*s13), ten(*s2))
    lg, ids = ten(4, 8, dtype=F32), i32(*range(8)).view(4, 2)
    so = i32(0, 2, 4)
    for call in (lambda: nv4.moe_balance_loss(lg, ids, seg_offsets=so, out=balance(1, 8)),
                 lambda: nv4.moe_balance_backward(lg, ids, balance(1, 8), ten(2, dtype=F32), seg_offsets=so),
                 lambda: nv4.moe_balance_backward(lg, ids, balance(2, 7), ten(2, dtype=F32), seg_offsets=so),
                 lambda: nv4.moe_balance_backward(lg, ids, balance(2, 8), ten(3, dtype=F32), seg_offsets=so),
                 lambda: nv4.moe_balance_backward(lg, ids, dtopk_w=ten(4, 3, dtype=F32)),
                 lambda: nv4.moe_balance_backward(lg, ids, dtopk_w=ten(4, 2, dtype=F32), out=ten(4, 9, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(4, 64), ten(8, 32), ids, ten(4, 2, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(4, 64), ten(8, 64), ids[:3], ten(3, 2, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(4, 64), ten(8, 64), ids, ten(4, 3, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(4, 128)[:, :64], ten(8, 64), ids, ten(4, 2, dtype=F32)),
                 lambda: nv4.moe_combine_backward(ten(4, 64), ten(8, 64), ids, ten(4, 2, dtype=F32), dY=ten(7, 64))):
        with pytest.raises(ValueError):
            call()
    assert not gpu.calls
