"""The MXFP4 binding on the CPU: what it passes to the library, on which stream, and what it
refuses.  A stand-in library records every call; tensors say that they are on a GPU, but live in
host memory, and streams are names.  No kernel runs, so a wrong stride, buffer or stream shows
here without touching memory that is not the call's."""

import contextlib
import types

import pytest
import torch

import nvfp4_w4a4_moe_amd as nv4
from nvfp4_w4a4_moe_amd import mxfp4

BF16 = torch.bfloat16


class OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0."""
    is_cuda = True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        Gpu.now.recorded.setdefault(self.data_ptr(), set()).add(stream.cuda_stream)


class Stream:
    def __init__(self, name, device="cpu"):
        self.cuda_stream, self.device = name, torch.device(device)

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream

    def __hash__(self):
        return hash(self.cuda_stream)

    def record_event(self, event=None):
        return event


class Gpu:
    """The stand-in: `calls` holds (function, arguments, the stream it was given, the current device),
    `made` the stream on which each tensor was allocated or copied, by address."""
    now = None

    def __init__(self, monkeypatch):
        Gpu.now = self
        self.calls, self.made, self.recorded, self.device = [], {}, {}, 0
        self.keep = []   # (no address is used twice)
        self.stream = Stream(100)
        empty, reshape = torch.empty, torch.Tensor.reshape

        def on_gpu(*shape, device=None, **k):
            t = empty(*shape, **k).as_subclass(OnGpu)
            self.made[t.data_ptr()] = self.stream.cuda_stream
            self.keep.append(t)
            return t

        @contextlib.contextmanager
        def stream(s):
            old, self.stream = self.stream, s
            dev, self.device = self.device, 0
            yield
            self.stream, self.device = old, dev

        @contextlib.contextmanager
        def device(d):
            old, self.device = self.device, 0 if isinstance(d, torch.device) else d
            yield
            self.device = old

        def copied(t, *shape):
            r = reshape(t, *shape)
            if r.data_ptr() != t.data_ptr():
                self.made[r.data_ptr()] = self.stream.cuda_stream
                self.keep.append(r)
            return r

        monkeypatch.setattr(torch, "empty", on_gpu)
        monkeypatch.setattr(OnGpu, "reshape", copied, raising=False)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: self.stream if d is not None or not self.device else Stream(900))
        monkeypatch.setattr(mxfp4, "_raw_stream", lambda i: self.stream.cuda_stream)
        monkeypatch.setattr(mxfp4, "load", lambda: self)
        monkeypatch.setattr(nv4, "load", lambda: self)

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 4096
        return lambda *a: self.calls.append((name, a[:-1], getattr(a[-1], "value", a[-1]), self.device)) or 0

    def args(self, name):
        return [a for n, a, *_ in self.calls if n == name]


@pytest.fixture
def gpu(monkeypatch):
    g = Gpu(monkeypatch)
    yield g
    Gpu.now = None


def ten(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def mx(rows, K):
    u8 = torch.uint8
    return nv4.MXFP4(ten(rows, K // 2, dtype=u8), ten(rows, nv4.mxfp4_scale_stride(K), dtype=u8), rows, K)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32).as_subclass(OnGpu)


def weights(E, H, I):
    return nv4.MXExpertWeights(mx(E * 2 * I, H), mx(E * H, I), E, H, I)


# ----------------------------------------------------------------------------- strides

# rows that overlap: one row repeated, and windows that share half of their elements
OVERLAPPING = [lambda n, dt: ten(1, 64, dtype=dt).expand(n, 64),
               lambda n, dt: ten((n + 1) * 32, dtype=dt).unfold(0, 64, 32)]


@pytest.mark.parametrize("make", OVERLAPPING)
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_rows_that_overlap_are_refused(gpu, make, dtype):
    """The library takes a matrix by its row stride.  A stride below the width is refused and
    never replaced by the width, which reads or writes rows that are not there."""
    w, lg, ok = weights(4, 64, 32), ten(3, 4, dtype=torch.float32), ten(3, 64, dtype=dtype)
    bad = make(3, dtype)
    for call in (lambda: nv4.mxfp4_quantize(bad),
                 lambda: nv4.mxfp4_quantize(bad, row_index=i32(0, 1, 2, 2)),
                 lambda: nv4.mxfp4_dequantize(mx(3, 64), out=bad),
                 lambda: nv4.mx_moe_few(bad, lg, w, 2),
                 lambda: nv4.mx_moe_few(ok, lg, w, 2, out=bad),
                 lambda: nv4.mxfp4_grouped_gemm(mx(3, 96), mx(64, 96), i32(0, 3), 1, 64, C=bad)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert not gpu.calls


def test_row_strides_are_the_tensors(gpu):
    wide = ten(5, 96)
    for x, ldx in ((wide, 96), (wide[:, :64], 96), (wide[::2, 32:], 192), (wide[:1, :64], 64), (ten(64).expand(1, 64), 64),
                   (ten(96, 1).t()[:, :64], 64)):
        nv4.mxfp4_quantize(x)
        assert gpu.args("mxfp4_quantize")[-1][5] == ldx
        nv4.mxfp4_dequantize(mx(*x.shape), out=x)
        assert gpu.args("mxfp4_dequantize")[-1][3] == ldx
        nv4.mxfp4_grouped_gemm(mx(x.shape[0], 96), mx(x.shape[1], 96), i32(0, 1), 1, x.shape[1], C=x)
        assert gpu.args("mxfp4_grouped_gemm")[-1][11] == ldx


@pytest.mark.parametrize("shape", [(2, 9, 64), (2, 7, 64), (2, 8, 65), (3, 8, 64), (16, 64)])
def test_weight_gradients_have_their_own_shape(gpu, shape):
    """Expert e's part of C starts e * A.rows rows in: a C with more rows would get them displaced."""
    o = dict(group_mode=nv4.NV4_GROUP_K)
    a, b, off = mx(8, 128), mx(64, 128), i32(0, 128, 128)
    with pytest.raises(ValueError, match=r"C must be \[2, 8, 64\]"):
        nv4.mxfp4_grouped_gemm(a, b, off, 2, 0, C=ten(*shape), **o)
    assert not gpu.calls
    assert nv4.mxfp4_grouped_gemm(a, b, off, 2, 0, C=ten(2, 8, 64), **o).shape == (2, 8, 64)
    assert gpu.args("mxfp4_grouped_gemm")[-1][11] == 64


# ----------------------------------------------------------------------------- devices

def test_scales_on_another_device_are_refused(gpu):
    """A tensor's codes and scales are both written or read by the kernel: both have to be there."""
    half = lambda rows, K: nv4.MXFP4(mx(rows, K).codes, torch.zeros(rows, nv4.mxfp4_scale_stride(K), dtype=torch.uint8),
                                     rows, K)
    x, seg = ten(4, 64), dict(nseg=1, seg_offsets=i32(0, 4), seg_padded_offsets=i32(0, 128))
    for call in (lambda: nv4.mxfp4_quantize(x, out=half(4, 64)),
                 lambda: nv4.mxfp4_quantize(x, layout=nv4.NV4_ROWS_AND_COLS, out=mx(64, 256), out_rows=half(4, 64), **seg),
                 lambda: nv4.mxfp4_dequantize(half(4, 64)),
                 lambda: nv4.mxfp4_grouped_gemm(mx(4, 64), mx(64, 64), i32(0, 4), 1, 32, epilogue=nv4.NV4_EPI_SWIGLU,
                                                q_out=half(4, 32), want_c=False)):
        with pytest.raises(ValueError, match="tensors on"):
            call()
    assert not gpu.calls


# ----------------------------------------------------------------------------- streams

def single_calls(stream):
    """Each call that makes its own outputs or workspace, as (call, its tensors)."""
    x, w, off, lg = ten(3, 64), weights(4, 64, 32), i32(0, 3), ten(3, 4, dtype=torch.float32)
    o = dict(stream=stream)
    both = dict(layout=nv4.NV4_ROWS_AND_COLS, seg_offsets=off, seg_padded_offsets=i32(0, 128))
    pair = lambda q: [q.codes, q.scales]
    return [lambda: pair(nv4.mxfp4_quantize(x, **o)),
            lambda: sum(map(pair, (lambda q: (q, q.rows_out))(nv4.mxfp4_quantize(x, **both, **o))), []),
            lambda: [nv4.mxfp4_dequantize(mx(3, 64), **o)], lambda: [nv4.mx_padded_offsets(off, **o)],
            lambda: [nv4.mxfp4_grouped_gemm(mx(3, 64), mx(32, 64), off, 1, 32, **o)],
            lambda: [nv4.mx_moe_few(x, lg, w, 2, **o)]]


@pytest.mark.parametrize("i", range(6))
def test_a_streams_call_takes_the_streams_memory(gpu, i):
    """A block of the current stream's pool may still be in use by kernels queued there, for which a
    call on another stream does not wait.  So outputs and workspaces come from the pool of the
    stream that writes them, and the outputs are kept from reuse until the caller's stream is done
    with them."""
    call = single_calls(Stream(200))[i]
    gpu.made.clear()
    outs = call()
    assert gpu.calls and {s for *_, s, _ in gpu.calls} == {200}
    assert gpu.made and set(gpu.made.values()) == {200}
    assert {t.data_ptr() for t in outs} == {a for a, s in gpu.recorded.items() if s == {100}} == set(gpu.recorded)
    assert gpu.stream == Stream(100)


@pytest.mark.parametrize("i", range(6))
@pytest.mark.parametrize("given", [None, 100])
def test_the_current_streams_call_stays_there(gpu, i, given):
    call = single_calls(given and Stream(given))[i]
    gpu.made.clear()
    call()
    assert {s for *_, s, _ in gpu.calls} == {100} == set(gpu.made.values()) and not gpu.recorded


T, E, K_, H, I = 3, 4, 2, 64, 32


def layer_tensors(b):
    """Every tensor of a layer's buffers."""
    for v in vars(b).values():
        if isinstance(v, torch.Tensor):
            yield v
        elif hasattr(v, "__dataclass_fields__"):
            yield from layer_tensors(v)


def forward(stream=None, bufs=None, n=T):
    return nv4.mx_moe_forward(ten(n, H), ten(n, E, dtype=torch.float32), weights(E, H, I), K_, bufs, stream=stream)


def backward(fwd, stream=None, bufs=None):
    wt = nv4.MXTransposedWeights(mx(E * I, H), mx(E * H, 2 * I))
    return nv4.mx_moe_backward(ten(T, H), fwd, wt, ten(T * K_, H), ten(T * K_, 2 * I), bufs, stream=stream)


LAYER_CALLS = {"mxfp4_quantize", "moe_permute", "mxfp4_grouped_gemm", "moe_combine", "mx_padded_offsets"}


@pytest.mark.parametrize("given", [None, 100, 200])
def test_a_layer_on_a_stream_takes_the_streams_memory(gpu, given):
    """Buffers that the layer makes (its routing among them) come from the pool of the stream that
    writes them, so that dropping them early gives them to that stream's later work only; those it
    returns wait for the caller's stream as well."""
    at = given or 100
    stream = given and Stream(given)
    kept = nv4.mx_alloc_forward(T, H, E, K_, I, keep_hact=True)
    gpu.made.clear()
    f = forward(stream)
    assert {n for n, *_ in gpu.calls} == LAYER_CALLS - {"mx_padded_offsets"} and {s for *_, s, _ in gpu.calls} == {at}
    mine = {t.data_ptr() for t in layer_tensors(f)}
    assert mine <= set(gpu.made) and set(gpu.made.values()) == {at}
    assert gpu.recorded == ({a: {100} for a in mine} if at == 200 else {})
    # buffers of the caller's stay as they are: only the routing is new
    gpu.made.clear(), gpu.recorded.clear()
    old = {t.data_ptr() for t in layer_tensors(kept)}
    f = forward(stream, kept)
    new = {t.data_ptr() for t in layer_tensors(f)} - old
    assert len(new) == 6 and new <= set(gpu.made) and set(gpu.made.values()) == {at}
    assert set(gpu.recorded) == (new if at == 200 else set())
    gpu.made.clear(), gpu.recorded.clear(), gpu.calls.clear()
    forward(stream, kept)   # routing and all: nothing is made
    assert not gpu.made and not gpu.recorded and {s for *_, s, _ in gpu.calls} == {at}
    gpu.calls.clear()
    g = backward(f, stream)
    assert {s for *_, s, _ in gpu.calls} == {at} == set(gpu.made.values())
    assert gpu.recorded == ({t.data_ptr(): {100} for t in layer_tensors(g)} if at == 200 else {})
    assert gpu.stream == Stream(100)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        forward(Stream(200, "cuda:1"))
    with pytest.raises(ValueError, match="stream of cuda:1"):
        backward(f, Stream(200, "cuda:1"))


def test_a_layer_refuses_host_tensors(gpu):
    with pytest.raises(ValueError, match="GPU"):
        nv4.mx_moe_forward(torch.zeros(T, H, dtype=BF16), torch.zeros(T, E), weights(E, H, I), K_)
    assert not gpu.calls and not gpu.made


@pytest.mark.parametrize("given", [None, 100, 200])
@pytest.mark.parametrize("transposed", [False, True])
def test_strided_weights_are_copied_on_the_stream(gpu, given, transposed):
    """Weights whose rows are not in one stride are copied first: on the stream that quantises them,
    which waits for no other."""
    stored = [ten(2 * I, E, H).transpose(0, 1), ten(H, E, I).transpose(0, 1)]
    at = given or 100
    quantize = nv4.mx_quantize_expert_weights_t if transposed else nv4.mx_quantize_expert_weights
    q = quantize(*stored, stream=given and Stream(given))
    tensors = [t for m in vars(q).values() if isinstance(m, nv4.MXFP4) for t in (m.codes, m.scales)]
    assert [s for *_, s, _ in gpu.calls] == [at] * 2
    copies = {a[0] for a in gpu.args("mxfp4_quantize")}
    assert copies | {t.data_ptr() for t in tensors} == set(gpu.made) and set(gpu.made.values()) == {at}
    assert set(gpu.recorded) == ({t.data_ptr() for t in tensors} if at == 200 else set())
    # contiguous weights are read where they are
    gpu.made.clear(), gpu.calls.clear()
    held = [ten(E, 2 * I, H), ten(E, H, I)]
    quantize(*held, stream=given and Stream(given))
    assert {a[0] for a in gpu.args("mxfp4_quantize")} == {t.data_ptr() for t in held}
    assert gpu.stream == Stream(100)


def test_a_layer_on_another_device_than_the_current_one(gpu):
    """Every call of the layer, moe_permute and moe_combine among them, runs with the tensors' device
    current and on that device's stream."""
    gpu.device = 1
    f = forward()
    backward(forward(None, nv4.mx_alloc_forward(T, H, E, K_, I, keep_hact=True)))
    nv4.mx_quantize_expert_weights(ten(E, 2 * I, H), ten(E, H, I))
    forward(Stream(200), f)
    assert LAYER_CALLS == {n for n, *_ in gpu.calls}
    assert {d for *_, d in gpu.calls} == {0} and {s for *_, s, _ in gpu.calls} == {100, 200}
    assert gpu.device == 1


# ----------------------------------------------------------------------------- shapes

def test_a_layers_inputs_fit_together(gpu):
    """Rows, experts and buffers of another batch: the routing would be written behind its buffers,
    or rows of x that do not exist be taken for others."""
    f32 = torch.float32
    fwd = lambda n=T, lg=(T, E), k=K_, h=H, bufs=None: nv4.mx_moe_forward(ten(n, h), ten(*lg, dtype=f32), weights(E, H, I),
                                                                          k, bufs)
    for lg in ((T + 1, E), (T - 1, E), (T, E + 1), (T * E,)):
        with pytest.raises(ValueError, match="logits"):
            fwd(lg=lg)
    with pytest.raises(ValueError, match="columns"):
        fwd(h=96)
    alloc = lambda n=T, h=H, k=K_: nv4.mx_alloc_forward(n, h, E, k, I, keep_hact=True)
    for other in (alloc(n=T + 1), alloc(k=1), alloc(k=3), alloc(h=96)):
        with pytest.raises(ValueError, match="bufs"):
            fwd(bufs=other)
    used = fwd(bufs=alloc())
    for field, n in (("topk_ids", (T, K_ + 1)), ("topk_ids", (T + 1, K_)), ("offsets", (E,))):
        bad = alloc()
        bad.routing = nv4.Routing(**{**vars(used.routing), field: ten(*n, dtype=torch.int32)})
        with pytest.raises(ValueError, match="bufs"):
            fwd(bufs=bad)
    with pytest.raises(ValueError, match="bufs"):
        strided = alloc()
        strided.out = ten(T, H + 8)[:, :H]
        fwd(bufs=strided)
    gpu.calls.clear()
    wt = nv4.MXTransposedWeights(mx(E * I, H), mx(E * H, 2 * I))
    for n in (T - 1, T + 1, 2 * T):
        with pytest.raises(ValueError, match="rows"):
            nv4.mx_moe_backward(ten(n, H), used, wt, ten(T * K_, H), ten(T * K_, 2 * I))
    for s13, s2 in (((E, 2 * I, H), (E, I, H)), ((E, 2 * I + 1, H), (E, H, I)), ((E, 2 * I, H), (E + 1, H, I))):
        for quantize in (nv4.mx_quantize_expert_weights, nv4.mx_quantize_expert_weights_t):
            with pytest.raises(ValueError, match="W2"):
                quantize(ten(*s13), ten(*s2))
    assert not gpu.calls


def test_weights_given_as_matrices(gpu):
    """W2 as [E*H, I], which its rows are in memory anyway."""
    for quantize in (nv4.mx_quantize_expert_weights, nv4.mx_quantize_expert_weights_t):
        gpu.calls.clear()
        quantize(ten(E, 2 * I, H), ten(E * H, I))
        assert sorted(a[3:5] for a in gpu.args("mxfp4_quantize")) == sorted([(E * 2 * I, H), (E * H, I)])
