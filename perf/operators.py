"""MXFP4 operators of the expert path: what they compute, on which inputs, at which sizes.

Three operators, each over the range in which a mixture-of-experts layer calls it:

  quantise   MXFP4 quantisation (OCP MX v1.0: blocks of 32 E2M1 codes under one E8M0
             power-of-two scale) along rows, or along the tokens of each expert for the
             operands of weight gradients.  The codes are returned as the values they
             stand for, which BF16 holds exactly.
  product    the grouped product of two MXFP4 operands: per expert rows . weights^T, with
             or without the SwiGLU epilogue, the weight gradients (contraction over an
             expert's tokens), and a linear layer's two gradients from BF16 inputs.
  few        a whole expert layer for a few tokens of a decode step: routing, quantised
             activations, gate and up products, SwiGLU, re-quantisation, down product and
             the weighted combine.

``run`` is the plain form in elementary torch operations (32 bits, rounded once to the
output's type) or, with ``own`` true, the calls of nvfp4_w4a4_moe_amd that a user makes.
``exact`` is the same definition in 64 bits, written apart from the plain form.

The layer of the larger cases is the one the benchmark and the tests use: hidden size
2048, 128 experts, eight per token, expert size 768.
"""

import math

import torch

own = False

BLOCK = 32        # elements under one scale
SEGMENT = 128     # an expert's token range is padded to this many columns
DEVICE = "cuda"
FP32, BF16 = "float32", "bfloat16"
MAX_EXACT_FLOPS = 1e14


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's activations before their first product
        dict(name="quantise_33_tokens", op="quantise", layout="rows", rows=33, cols=2048, dtype=BF16),
        # the learner batch's activations: 8 sequences of 8192 tokens
        dict(name="quantise_learner_tokens", op="quantise", layout="rows", rows=65536, cols=2048, dtype=BF16),
        # a weight gradient's operand: tokens gathered into expert order, blocks down the tokens
        dict(name="quantise_by_expert", op="quantise", layout="tokens", rows=16384, cols=2048, dtype=BF16, experts=128,
             k=8, skew=1.1),
        # FP32 gradients of an odd number of rows with an odd number of blocks
        dict(name="quantise_fp32_odd", op="quantise", layout="rows", rows=9973, cols=1056, dtype=FP32),
        # one dense product at the benchmark's shape
        dict(name="product_dense", op="product", form="rows", tokens=8192, k=1, experts=1, K=2048, N=768, gather=False,
             epilogue="none", out=BF16, skew=0.0),
        # a decode batch's gate and up projection: a few rows for each of many experts
        dict(name="product_decode_swiglu", op="product", form="rows", tokens=96, k=8, experts=128, K=2048, N=768,
             gather=True, epilogue="swiglu", out=BF16, skew=0.0),
        # gate and up projection of 16384 tokens with skewed expert loads
        dict(name="product_swiglu", op="product", form="rows", tokens=16384, k=8, experts=128, K=2048, N=768,
             gather=True, epilogue="swiglu", out=BF16, skew=1.1),
        # down projection with FP32 rows for the combine, ragged expert loads
        dict(name="product_down_ragged", op="product", form="rows", tokens=10007, k=2, experts=8, K=768, N=2048,
             gather=False, epilogue="none", out=FP32, skew=0.7),
        # a linear layer's gradients from BF16 rows: quantisation both ways and both products
        dict(name="product_gradients", op="product", form="gradients", tokens=4096, k=8, experts=64, K=2048, N=768,
             skew=0.7),
        # one token: latency and the bytes of eight experts
        dict(name="few_1", op="few", tokens=1, k=8, experts=128, H=2048, I=768),
        # a handful of sequences
        dict(name="few_7", op="few", tokens=7, k=8, experts=128, H=2048, I=768),
        # a full decode batch: nearly every expert is read
        dict(name="few_64", op="few", tokens=64, k=8, experts=128, H=2048, I=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "few"])
    if op == "quantise":
        cols = BLOCK * _log(rng, 2, 160)
        dtype = rng.choice([BF16, FP32])
        if rng.random() < 0.5:
            rows = min(_log(rng, 1, 65536), 65536 * 2048 // (cols if dtype == BF16 else 2 * cols))
            return dict(op=op, layout="rows", rows=rows, cols=cols, dtype=dtype)
        experts = _log(rng, 1, 256)
        k = rng.randint(1, min(8, experts))
        rows = min(_log(rng, 1, 16384), 16384 * 8 * 2048 // (k * cols))
        return dict(op=op, layout="tokens", rows=rows, cols=cols, dtype=dtype, experts=experts, k=k,
                    skew=round(rng.uniform(0.0, 1.2), 2))
    experts = _log(rng, 2, 256)
    k = rng.randint(1, min(8, experts))
    if op == "few":
        H, I = BLOCK * _log(rng, 4, 128), BLOCK * _log(rng, 2, 44)
        experts = max(2, min(experts, 128 * 768 * 2048 // (H * I)))
        k = min(k, experts)
        tokens = min(rng.randint(1, 64), 64 * 8 * 768 * 2048 // (k * H * I))
        return dict(op=op, tokens=tokens, k=k, experts=experts, H=H, I=I)
    form = rng.choice(["rows", "rows", "gradients"])
    K, N = BLOCK * _log(rng, 2, 100), BLOCK * _log(rng, 2, 64)
    experts = max(2, min(experts, 128 * 768 * 2048 // (K * N)))
    k = min(k, experts)
    skew = round(rng.uniform(0.0, 1.2), 2)
    tokens = max(1, min(_log(rng, 1, 16384), 8 * 16384 * 2048 * 768 // (2 * k * K * N), 16384 * 8 * 2048 // (k * max(K, N))))
    if form == "gradients":
        experts = max(k, 2, min(experts, 64 * 768 * 2048 // (K * N)))
        tokens = max(1, min(tokens // 2, 4096 * 8 * 2048 // (k * max(K, N))))
        return dict(op=op, form=form, tokens=tokens, k=k, experts=experts, K=K, N=N, skew=skew)
    N -= rng.choice([0, 0, rng.randint(1, BLOCK - 1)])       # output columns need not be whole blocks
    return dict(op=op, form=form, tokens=tokens, k=k, experts=experts, K=K, N=N, gather=rng.random() < 0.5,
                epilogue=rng.choice(["none", "swiglu"]), out=rng.choice([BF16, FP32]), skew=skew)


# ------------------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEVICE) * std


def _activations(g, rows, cols, dtype):
    """N(0, 1) with one value in a thousand twenty times as large, as the tests draw them."""
    x = _normal(g, rows, cols)
    x = torch.where(torch.rand(rows, cols, generator=g, device=DEVICE) < 1e-3, x * 20, x)
    return x.to(getattr(torch, dtype))


def _pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def _codes_and_scales(x):
    """MXFP4 of the last dimension of an FP32 tensor: (E2M1 codes, E8M0 bytes)."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1)
    _, e = torch.frexp(amax)                                 # amax = m 2^e with m in [0.5, 1)
    e8 = torch.where(amax > 0, e - 3 + 127, torch.zeros_like(e)).clamp(0, 254).int()
    inv = ((254 - e8) << 23).view(torch.float32)             # 2^(127 - e8): exact
    y = b.abs() * inv[..., None]
    c = (y > 0.25).to(torch.uint8)                           # ties go to the even code
    for_even, for_odd = (1.25, 2.5, 5.0), (0.75, 1.75, 3.5)
    c += (y >= for_odd[0]).to(torch.uint8) + (y > for_even[0]).to(torch.uint8) + (y >= for_odd[1]).to(torch.uint8)
    c += (y > for_even[1]).to(torch.uint8) + (y >= for_odd[2]).to(torch.uint8) + (y > for_even[2]).to(torch.uint8)
    c |= torch.signbit(b).to(torch.uint8) << 3
    return c.reshape(x.shape), e8.to(torch.uint8)


def _packed(x):
    """What a program keeps of a quantised matrix: packed codes [rows, K/2] and the scale
    bytes [rows, K/32 rounded up to 4] with zeros behind the last block."""
    c, s = _codes_and_scales(x.float())
    s = torch.nn.functional.pad(s, (0, -s.shape[-1] % 4))
    return dict(codes=_pack(c), scales=s.contiguous(), rows=x.shape[0], K=x.shape[1])


def _route(g, case, tokens):
    """The routing a program has in hand: each expert's rows by token.  The experts' loads
    are the case's own (Gumbel top-k of Zipf-like logits), which tokens make them up is the
    seed's."""
    E, k, skew = case["experts"], case["k"], case["skew"]
    loads = torch.Generator(device=DEVICE)
    loads.manual_seed(E * 1000 + k)
    rank = torch.randperm(E, generator=loads, device=DEVICE).float() + 1
    u = torch.rand(tokens, E, generator=loads, device=DEVICE).clamp(1e-7, 1 - 1e-7)
    ids = (-skew * rank.log() - (-u.log()).log()).topk(k, dim=1).indices
    flat = ids[torch.randperm(tokens, generator=g, device=DEVICE)].reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    zero = torch.zeros(1, dtype=torch.int64, device=DEVICE)
    offsets = torch.cat([zero, counts.cumsum(0)])
    padded = torch.cat([zero, ((counts + SEGMENT - 1) // SEGMENT * SEGMENT).cumsum(0)])
    expert = flat[order]
    slot = padded[expert] + torch.arange(flat.numel(), device=DEVICE) - offsets[expert]
    return dict(row_token=(order // k).int(), offsets=offsets.int(), padded=padded.int(), slot=slot,
                sizes=counts.tolist(), columns=int(padded[-1]))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantise":
        s["x"] = _activations(g, case["rows"], case["cols"], case["dtype"])
        if case["layout"] == "tokens":
            s |= _route(g, case, case["rows"])
        return s
    T, E = case["tokens"], case["experts"]
    if case["op"] == "few":
        H, I = case["H"], case["I"]
        s["x"] = _activations(g, T, H, BF16)
        s["logits"] = _normal(g, T, E)
        s["w13"] = _packed(_normal(g, E * 2 * I, H, std=0.02).bfloat16())
        s["w2"] = _packed(_normal(g, E * H, I, std=0.02).bfloat16())
        return s
    K, N = case["K"], case["N"]
    s |= _route(g, case, T)
    R = T * case["k"]
    if case["form"] == "gradients":
        s["x"] = _activations(g, T, K, BF16)
        s["dy"] = _normal(g, R, N, std=1e-3).bfloat16()
        s["wt"] = _packed(_normal(g, E * K, N, std=0.02).bfloat16())      # per expert [K][N]: laid out once a step
        return s
    s["a"] = _packed(_activations(g, T if case["gather"] else R, K, BF16))
    s["b"] = _packed(_normal(g, E * N * (2 if case["epilogue"] == "swiglu" else 1), K, std=0.02).bfloat16())
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"quantise": _plain_quantise, "product": _plain_product, "few": _plain_few}[state["op"]](state)


def _run_own(s):
    import nvfp4_w4a4_moe_amd as nv4
    mx = lambda q: nv4.MXFP4(q["codes"], q["scales"], q["rows"], q["K"])
    if s["op"] == "quantise":
        if s["layout"] == "rows":
            return nv4.mxfp4_dequantize(nv4.mxfp4_quantize(s["x"]))
        padded = nv4.mx_padded_offsets(s["offsets"])
        q = nv4.mxfp4_quantize(s["x"], layout=nv4.NV4_COLS, nseg=s["experts"], seg_offsets=s["offsets"],
                               seg_padded_offsets=padded, row_index=s["row_token"])
        return nv4.mxfp4_dequantize(q)[:, :s["columns"]]
    if s["op"] == "few":
        w = nv4.MXExpertWeights(mx(s["w13"]), mx(s["w2"]), s["experts"], s["H"], s["I"])
        return nv4.mx_moe_few(s["x"], s["logits"], w, s["k"])
    E, R = s["experts"], s["row_token"].numel()
    if s["form"] == "rows":
        epilogue = nv4.NV4_EPI_SWIGLU if s["epilogue"] == "swiglu" else nv4.NV4_EPI_NONE
        return nv4.mxfp4_grouped_gemm(mx(s["a"]), mx(s["b"]), s["offsets"], E, s["N"], M_cap=R,
                                      a_rows=s["row_token"] if s["gather"] else None, epilogue=epilogue,
                                      out_dtype=getattr(torch, s["out"]))
    padded = nv4.mx_padded_offsets(s["offsets"])
    seg = dict(nseg=E, seg_offsets=s["offsets"], seg_padded_offsets=padded)
    dyc = nv4.mxfp4_quantize(s["dy"], layout=nv4.NV4_ROWS_AND_COLS, **seg)
    xc = nv4.mxfp4_quantize(s["x"], layout=nv4.NV4_COLS, row_index=s["row_token"], **seg)
    dx = nv4.mxfp4_grouped_gemm(dyc.rows_out, mx(s["wt"]), s["offsets"], E, s["K"], M_cap=R, out_dtype=torch.bfloat16)
    dw = nv4.mxfp4_grouped_gemm(dyc, xc, padded, E, 0, group_mode=nv4.NV4_GROUP_K)
    return dict(dx=dx, dw=dw)


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_PAIRS = {}


def _pairs():
    """The two E2M1 values of every byte."""
    if not _PAIRS:
        v = torch.tensor(_MAGNITUDES + tuple(-m for m in _MAGNITUDES), device=DEVICE)
        byte = torch.arange(256, device=DEVICE)
        _PAIRS[0] = torch.stack([v[byte & 15], v[byte >> 4]], -1)
    return _PAIRS[0]


def _power(e8):
    """2^(e8 - 127) as FP32, exact (2^-127 is subnormal)."""
    bits = torch.where(e8 == 0, torch.full_like(e8, 1 << 22, dtype=torch.int32), e8.int() << 23)
    return bits.view(torch.float32)


def _values(codes, scales):
    v = torch.nn.functional.embedding(codes.int(), _pairs()).flatten(-2)
    blocks = v.shape[-1] // BLOCK
    return (v.unflatten(-1, (blocks, BLOCK)) * _power(scales[..., :blocks])[..., None]).flatten(-2)


def _rounded(x):
    """The MXFP4 values nearest to x, FP32."""
    c, e8 = _codes_and_scales(x)
    m = _pairs()[:16, 0][c.int()]
    return (m.unflatten(-1, (-1, BLOCK)) * _power(e8)[..., None]).flatten(-2)


def _by_expert(s, x):
    """Rows in expert order at their padded positions, zeros between: [columns, cols]."""
    out = torch.zeros(s["columns"], x.shape[1], device=DEVICE)
    out[s["slot"]] = x.float()
    return out


def _plain_quantise(s):
    if s["layout"] == "rows":
        return _rounded(s["x"].float()).bfloat16()
    return _rounded(_by_expert(s, s["x"][s["row_token"]]).t().contiguous()).bfloat16()


def _grouped(a, b, sizes):
    """Rows of expert e (sizes[e] of them) times b[e]^T: one product per expert, all large."""
    out = torch.empty(a.shape[0], b.shape[1], device=DEVICE)
    at = 0
    for e, n in enumerate(sizes):
        torch.mm(a[at:at + n], b[e].t(), out=out[at:at + n])
        at += n
    return out


def _silu_up(y):
    gate, up = y.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_product(s):
    E = s["experts"]
    if s["form"] == "rows":
        a = _values(s["a"]["codes"], s["a"]["scales"])
        if s["gather"]:
            a = a[s["row_token"]]
        b = _values(s["b"]["codes"], s["b"]["scales"])
        y = _grouped(a, b.unflatten(0, (E, -1)), s["sizes"])
        if s["epilogue"] == "swiglu":
            y = _silu_up(y)
        return y.to(getattr(torch, s["out"]))
    wt = _values(s["wt"]["codes"], s["wt"]["scales"]).unflatten(0, (E, -1))
    dx = _grouped(_rounded(s["dy"].float()), wt, s["sizes"]).bfloat16()
    dyc = _rounded(_by_expert(s, s["dy"]).t().contiguous())
    xc = _rounded(_by_expert(s, s["x"][s["row_token"]]).t().contiguous())
    dw = torch.zeros(E, s["N"], s["K"], device=DEVICE)
    at = 0
    for e, n in enumerate(s["sizes"]):
        n = (n + SEGMENT - 1) // SEGMENT * SEGMENT
        torch.mm(dyc[:, at:at + n], xc[:, at:at + n].t(), out=dw[e])
        at += n
    return dict(dx=dx, dw=dw)


def _plain_few(s):
    T, k, E, H, I = s["tokens"], s["k"], s["experts"], s["H"], s["I"]
    p = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    ids = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k]
    weight = p.gather(1, ids)
    flat = ids.reshape(-1)
    of = lambda q, rows: _values(q["codes"].unflatten(0, (E, rows))[flat], q["scales"].unflatten(0, (E, rows))[flat])
    x = _rounded(s["x"].float()).repeat_interleave(k, 0)
    h = _rounded(_silu_up(torch.matmul(of(s["w13"], 2 * I), x[..., None])[..., 0]))
    y = torch.matmul(of(s["w2"], H), h[..., None])[..., 0]
    return (y.view(T, k, H) * weight[..., None]).sum(1).bfloat16()


# ------------------------------------------------------------------------------ 64 bits

def _exact_power(e):
    """2^e in 64 bits from a table (pow rounds)."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=DEVICE)[e.long() + 160]


def _exact_mx(x):
    """MXFP4 values of the last dimension in 64 bits: round |x| / 2^e to the E2M1 grid's
    step of its binade, halves to even."""
    b = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = torch.where(_exact_power(e) > amax, e - 1, e)
    e = torch.where(_exact_power(e + 1) <= amax, e + 1, e)
    scale = _exact_power((e - 2).clamp(-127, 127))
    y = (b / scale).abs().clamp(max=6.0)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    q = (torch.round(y / step) * step).clamp(max=6.0) * torch.sign(b) * scale
    return torch.where(amax > 0, q, torch.zeros_like(q)).reshape(x.shape)


def _exact_values(q):
    low, high = (q["codes"] & 15).long(), (q["codes"] >> 4).long()
    c = torch.stack([low, high], -1).flatten(-2)
    m = c & 7
    mag = torch.where(m < 2, m * 0.5, _exact_power((m // 2 - 1).clamp(min=0)) * (1 + 0.5 * (m % 2)))
    v = torch.where(c > 7, -mag, mag)
    n = q["K"] // BLOCK
    scale = _exact_power(q["scales"][:, :n].long() - 127)
    return (v.reshape(q["rows"], n, BLOCK) * scale[..., None]).reshape(q["rows"], q["K"])


def exact(case, seed):
    w = work(case)
    if w["flops"] > MAX_EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if case["op"] == "quantise":
        if case["layout"] == "rows":
            return _exact_mx(s["x"])
        out = torch.zeros(case["cols"], s["columns"], dtype=torch.float64, device=DEVICE)
        for e in range(case["experts"]):
            lo, hi = sum(s["sizes"][:e]), sum(s["sizes"][:e + 1])
            at, n = int(s["padded"][e]), -(-(hi - lo) // BLOCK) * BLOCK
            rows = torch.zeros(n, case["cols"], dtype=torch.float64, device=DEVICE)
            rows[:hi - lo] = s["x"][s["row_token"][lo:hi].long()].double()
            if n:
                out[:, at:at + n] = _exact_mx(rows.t().contiguous())
        return out
    E = case["experts"]
    if case["op"] == "few":
        H, I, k = case["H"], case["I"], case["k"]
        p = torch.softmax(s["logits"].double(), 1)
        x = _exact_mx(s["x"])
        out = torch.zeros(case["tokens"], H, dtype=torch.float64, device=DEVICE)
        chosen = s["logits"].topk(k, dim=1).indices
        for e in sorted(set(chosen.reshape(-1).tolist())):
            part = lambda q, n: _exact_values(dict(codes=q["codes"][e * n:(e + 1) * n], K=q["K"], rows=n,
                                                   scales=q["scales"][e * n:(e + 1) * n]))
            t = (chosen == e).any(1).nonzero()[:, 0]
            y = x[t] @ part(s["w13"], 2 * I).t()
            h = _exact_mx(y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:])
            out[t] += p[t, e][:, None] * (h @ part(s["w2"], H).t())
        return out
    ends = [sum(s["sizes"][:e]) for e in range(E + 1)]
    if case["form"] == "rows":
        a, b = _exact_values(s["a"]), _exact_values(s["b"]).reshape(E, -1, case["K"])
        if case["gather"]:
            a = a[s["row_token"].long()]
        y = torch.cat([a[ends[e]:ends[e + 1]] @ b[e].t() for e in range(E)])
        if case["epilogue"] == "swiglu":
            N = case["N"]
            y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
        return y
    wt = _exact_values(s["wt"]).reshape(E, case["K"], case["N"])
    dy, dws = _exact_mx(s["dy"]), []
    dx = torch.cat([dy[ends[e]:ends[e + 1]] @ wt[e].t() for e in range(E)])
    for e in range(E):
        n = s["sizes"][e]
        pad = lambda v: _exact_mx(torch.nn.functional.pad(v.double().t(), (0, -n % BLOCK)).contiguous())
        rows = slice(ends[e], ends[e + 1])
        dws.append(pad(s["dy"][rows]) @ pad(s["x"][s["row_token"][rows].long()]).t() if n else
                   torch.zeros(case["N"], case["K"], dtype=torch.float64, device=DEVICE))
    return dict(dx=dx, dw=torch.stack(dws))


# ------------------------------------------------------------------------------ floors

def _mx_bytes(rows, K):
    return rows * (K // 2 + K // BLOCK)


def _experts_read(tokens, k, experts):
    """Experts that some token chooses, on average over even routing."""
    return experts * (1 - (1 - k / experts) ** tokens)


def work(case):
    size = {BF16: 2, FP32: 4}
    if case["op"] == "quantise":
        n = case["rows"] * case["cols"]
        out = n * case.get("k", 1)
        return dict(bytes=n * size[case["dtype"]] + out * 2 + (4 * case["rows"] * case["k"] if "k" in case else 0),
                    flops=4 * out)
    T, k, E = case["tokens"], case["k"], case["experts"]
    R = T * k
    if case["op"] == "few":
        H, I = case["H"], case["I"]
        read = _experts_read(T, k, E)
        return dict(bytes=int(read * (_mx_bytes(2 * I, H) + _mx_bytes(H, I))) + T * (2 * H + 4 * E + 2 * H),
                    flops=2 * R * 3 * H * I)
    K, N = case["K"], case["N"]
    read = _experts_read(T, k, E)
    if case["form"] == "gradients":
        return dict(bytes=2 * R * N + 2 * T * K + 4 * R + int(read * _mx_bytes(K, N)) + 2 * R * K + 4 * E * N * K,
                    flops=4 * R * N * K)
    n = N * (2 if case["epilogue"] == "swiglu" else 1)
    a = _mx_bytes(T, K) + 4 * R if case["gather"] else _mx_bytes(R, K)
    return dict(bytes=a + int(read * _mx_bytes(n, K)) + R * N * size[case["out"]], flops=2 * R * n * K)
