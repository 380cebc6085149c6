"""FP8 operators of the expert path and the training side of its router: what they compute, on
which inputs, at which sizes.

Four operators, each over the range in which a mixture-of-experts layer calls it:

  quantise   FP8 (E4M3) quantisation with an FP32 scale for each block of 128: along rows, along
             the tokens of each expert, both from one read, or in 128 x 128 blocks of weights.
             The codes are returned as the values they stand for.
  product    the grouped product of two such operands: per expert rows . weights^T, with or
             without the SwiGLU epilogue and its re-quantisation, and a linear layer's two
             gradients from BF16 rows (the data gradient through the transposed weights, the
             weight gradient over an expert's tokens).
  balance    the router's balance and z losses with per-expert counts, and the gradient of the
             logits (of both losses and of the routing weights).
  combine    the gradients of the weighted sum of each token's expert rows.

``run`` is the plain form in elementary torch operations (32 bits, rounded once to the output's
type) or, with ``own`` true, the calls of nvfp4_w4a4_moe_amd that a user makes.  ``exact`` is the
same definition in 64 bits, written apart from the plain form.

The layer of the larger cases is the one the benchmark and the tests use: hidden size 2048,
128 experts, eight per token, expert size 768.
"""

import math

import torch

own = False

BLOCK = 128       # elements under one scale, and the columns to which an expert's tokens are padded
DEVICE = "cuda"
FP32, BF16 = "float32", "bfloat16"
MAX_EXACT_FLOPS = 1e14


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's activations before their first product
        dict(name="quantise_33_tokens", op="quantise", layout="rows", rows=33, cols=2048, dtype=BF16, pow2=False),
        # the upstream gradients of the gate and up rows: along rows for the data gradient, along each
        # expert's tokens for the weight gradient
        dict(name="quantise_both", op="quantise", layout="both", rows=131072, cols=1536, dtype=BF16, experts=128, k=8,
             skew=1.1, pow2=False),
        # one dense product at the benchmark's shape
        dict(name="product_dense", op="product", form="rows", tokens=8192, k=1, experts=1, K=2048, N=768, gather=False,
             epilogue="none", out=BF16, skew=0.0, pow2=False),
        # one token's gate and up projection: a row for each of eight experts
        dict(name="product_token", op="product", form="rows", tokens=1, k=8, experts=128, K=2048, N=768, gather=True,
             epilogue="swiglu", out=BF16, skew=0.0, pow2=False),
        # a decode batch's gate and up projection: a few rows for each of many experts
        dict(name="product_decode_swiglu", op="product", form="rows", tokens=96, k=8, experts=128, K=2048, N=768,
             gather=True, epilogue="swiglu", out=BF16, skew=0.0, pow2=False),
        # gate and up projection of 16384 tokens with skewed expert loads, its result re-quantised for
        # the down projection
        dict(name="product_swiglu", op="product", form="rows", tokens=16384, k=8, experts=128, K=2048, N=768,
             gather=True, epilogue="requantise", out=BF16, skew=1.1, pow2=False),
        # down projection with FP32 rows for the combine: ragged expert loads, a last block of 80, an odd
        # number of columns
        dict(name="product_down_ragged", op="product", form="rows", tokens=10007, k=2, experts=8, K=720, N=2047,
             gather=False, epilogue="none", out=FP32, skew=0.7, pow2=False),
        # a linear layer's gradients from BF16 rows: quantisation both ways and both products
        dict(name="product_gradients", op="product", form="gradients", tokens=4096, k=8, experts=64, K=2048, N=768,
             skew=0.7, pow2=False),
        # a short batch's losses, some of its tokens padding, with the gradient of the logits
        dict(name="balance_short", op="balance", tokens=257, experts=60, k=4, sequences=3, padding=0.2, renorm=True),
        # the learner batch: eight sequences of 8192 tokens, a loss for each
        dict(name="balance_learner", op="balance", tokens=65536, experts=128, k=8, sequences=8, padding=0.0,
             renorm=False),
        # a few tokens' gradients of FP32 expert rows
        dict(name="combine_33_tokens", op="combine", tokens=33, H=2048, k=8, rows=FP32, out=FP32),
        # a training batch's gradients of BF16 expert rows
        dict(name="combine_training", op="combine", tokens=16384, H=2048, k=8, rows=BF16, out=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "balance", "combine"])
    if op == "balance":
        experts = _log(rng, 2, 512)
        tokens = min(_log(rng, 1, 65536), 65536 * 128 // experts)
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(8, experts)),
                    sequences=rng.choice([1, rng.randint(1, 40)]), padding=round(rng.choice([0.0, rng.uniform(0, 0.9)]), 2),
                    renorm=rng.random() < 0.5)
    if op == "combine":
        k, H = rng.randint(1, 8), 4 * _log(rng, 8, 2048)
        return dict(op=op, tokens=max(1, min(_log(rng, 1, 16384), 16384 * 8 * 2048 // (2 * k * H))), H=H, k=k,
                    rows=rng.choice([BF16, FP32]), out=rng.choice([BF16, FP32]))
    pow2 = rng.random() < 0.3
    if op == "quantise":
        layout = rng.choice(["rows", "tokens", "both", "tiles"])
        cols, dtype = 16 * _log(rng, 2, 320), rng.choice([BF16, FP32])
        most = 131072 * 1536 // (cols if dtype == BF16 else 2 * cols)
        if layout == "rows":
            return dict(op=op, layout=layout, rows=min(_log(rng, 1, 131072), most), cols=cols, dtype=dtype, pow2=pow2)
        experts = _log(rng, 1, 256)
        if layout == "tiles":
            return dict(op=op, layout=layout, rows=experts * max(1, min(_log(rng, 1, 2048), most // (2 * experts))),
                        cols=cols, dtype=dtype, experts=experts, pow2=pow2)
        k = rng.randint(1, min(8, experts))
        tokens = max(1, min(_log(rng, 1, 16384), most // (2 * k)))
        rows = tokens if layout == "tokens" else tokens * k
        return dict(op=op, layout=layout, rows=rows, cols=cols, dtype=dtype, experts=experts, k=k,
                    skew=round(rng.uniform(0.0, 1.2), 2), pow2=pow2)
    experts = _log(rng, 2, 256)
    k = rng.randint(1, min(8, experts))
    form = rng.choice(["rows", "rows", "gradients"])
    K, N = 16 * _log(rng, 4, 200), 32 * _log(rng, 2, 64)
    experts = max(2, min(experts, 128 * 768 * 2048 // (K * N)))
    k = min(k, experts)
    skew = round(rng.uniform(0.0, 1.2), 2)
    tokens = max(1, min(_log(rng, 1, 16384), 8 * 16384 * 2048 * 768 // (2 * k * K * N), 16384 * 8 * 2048 // (k * max(K, N))))
    if form == "gradients":
        experts = max(k, 2, min(experts, 64 * 768 * 2048 // (K * N)))
        tokens = max(1, min(tokens // 2, 4096 * 8 * 2048 // (k * max(K, N))))
        return dict(op=op, form=form, tokens=tokens, k=k, experts=experts, K=K, N=N, skew=skew, pow2=pow2)
    epilogue = rng.choice(["none", "swiglu", "requantise"])
    if epilogue == "none":
        N -= rng.choice([0, 0, rng.randint(1, 31)])          # plain output columns come in any number
    return dict(op=op, form=form, tokens=tokens, k=k, experts=experts, K=K, N=N, gather=rng.random() < 0.5,
                epilogue=epilogue, out=BF16 if epilogue == "requantise" else rng.choice([BF16, FP32]), skew=skew,
                pow2=pow2)


# ------------------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEVICE) * std


def _activations(g, rows, cols, dtype):
    """N(0, 1) with one value in a thousand twenty times as large, as the tests draw them."""
    x = _normal(g, rows, cols)
    x = torch.where(torch.rand(rows, cols, generator=g, device=DEVICE) < 1e-3, x * 20, x)
    return x.to(getattr(torch, dtype))


def _quotient(a, b):
    """a / b correctly rounded to FP32: the 64-bit quotient of two FP32 numbers, rounded."""
    return torch.div(torch.full_like(b, a, dtype=torch.float64), b.double()).float()


def _scale(amax, pow2):
    """(S, G) of blocks with these largest magnitudes: what multiplies a value before it is
    rounded, and the scale that is kept."""
    if pow2:
        m, e = torch.frexp(amax)                             # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
        t = (9 - e - (m > 0.875).int()).clamp(max=126)
        S = ((t.clamp(min=-126) + 127).int() << 23).view(torch.float32)
    else:
        S = _quotient(448.0, amax).clamp(max=2.0 ** 126)
    S = torch.where(amax > 0, S, torch.ones_like(S))
    return S, _quotient(1.0, S)


def _codes(x, pow2):
    """E4M3 codes (as torch's type) and scales of blocks of 128 along the last dimension of an FP32
    tensor; the last block may be shorter."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    S, G = _scale(b.abs().amax(-1), pow2)
    return (b * S[..., None]).flatten(-2)[..., :K].to(torch.float8_e4m3fn), G


def _tiles(x, experts, pow2):
    """The same in 128 x 128 blocks of each of `experts` stacked matrices: codes [experts, m, K],
    scales [experts, m / 128, K / 128] (rounded up)."""
    m, K = x.shape[0] // experts, x.shape[1]
    b = torch.nn.functional.pad(x.view(experts, m, K), (0, -K % BLOCK, 0, -m % BLOCK))
    b = b.unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))            # [experts, rows, 128, columns, 128]
    S, G = _scale(b.abs().amax((2, 4)), pow2)
    q = (b * S[:, :, None, :, None]).flatten(3, 4).flatten(1, 2)[:, :m, :K]
    return q.to(torch.float8_e4m3fn), G


def _kept(codes, scales, rows, K, experts=0):
    """What a program keeps of a quantised matrix."""
    return dict(codes=codes.reshape(rows, K).contiguous().view(torch.uint8), scales=scales.contiguous(), rows=rows, K=K,
                experts=experts)


def _route(g, case, tokens):
    """The routing a program has in hand: each expert's rows by token.  The experts' loads are the
    case's own (Gumbel top-k of Zipf-like logits), which tokens make them up is the seed's."""
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
    padded = torch.cat([zero, ((counts + BLOCK - 1) // BLOCK * BLOCK).cumsum(0)])
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
        if case["layout"] == "both":
            s |= _route(g, case, case["rows"] // case["k"])
        elif case["layout"] == "tokens":
            s |= _route(g, case, case["rows"])
        return s
    T, k = case["tokens"], case["k"]
    if case["op"] == "combine":
        H = case["H"]
        s["y"] = _normal(g, T * k, H).to(getattr(torch, case["rows"]))
        s["dout"] = _normal(g, T, H, std=1e-3).to(getattr(torch, case["out"]))
        s["topk_w"] = torch.softmax(_normal(g, T, k), 1)
        s["token_row"] = torch.randperm(T * k, generator=g, device=DEVICE).int().view(T, k)
        return s
    E = case["experts"]
    if case["op"] == "balance":
        s["logits"] = _normal(g, T, E, std=1.5) + _normal(g, E)
        order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices
        s["topk_ids"] = order[:, :k].int().contiguous()
        s["dtopk_w"] = _normal(g, T, k, std=1e-3)
        cuts = torch.randint(0, T + 1, (case["sequences"] - 1,), generator=g, device=DEVICE).sort().values
        ends = torch.tensor([0, T], device=DEVICE)
        s["seq_offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).int()
        s["mask"] = torch.rand(T, generator=g, device=DEVICE) >= case["padding"] if case["padding"] else None
        s["dloss"] = torch.tensor([1e-2, 1e-3], device=DEVICE)
        return s
    K, N = case["K"], case["N"]
    s |= _route(g, case, T)
    R = T * k
    if case["form"] == "gradients":
        s["x"] = _activations(g, T, K, BF16)
        s["dy"] = _normal(g, R, N, std=1e-3).bfloat16()
        w = _normal(g, E * N, K, std=0.02).bfloat16().float()
        codes, scales = _tiles(w, E, case["pow2"])           # the forward's weights, transposed once a step
        s["wt"] = _kept(codes.transpose(1, 2), scales.transpose(1, 2), E * K, N, E)
        return s
    rows = T if case["gather"] else R
    s["a"] = _kept(*_codes(_activations(g, rows, K, BF16).float(), case["pow2"]), rows, K)
    n = N * (1 if case["epilogue"] == "none" else 2)
    w = _normal(g, E * n, K, std=0.02).bfloat16().float()
    s["b"] = _kept(*_tiles(w, E, case["pow2"]), E * n, K, E)
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"quantise": _plain_quantise, "product": _plain_product, "balance": _plain_balance,
            "combine": _plain_combine}[state["op"]](state)


def _run_own(s):
    import nvfp4_w4a4_moe_amd as nv4
    if s["op"] == "balance":
        b = nv4.moe_balance_loss(s["logits"], s["topk_ids"], mask=s["mask"], seg_offsets=s["seq_offsets"])
        dlogits = nv4.moe_balance_backward(s["logits"], s["topk_ids"], b, s["dloss"], dtopk_w=s["dtopk_w"],
                                           mask=s["mask"], seg_offsets=s["seq_offsets"],
                                           flags=nv4.NV4_RENORM if s["renorm"] else 0)
        return dict(loss=b.loss, counts=b.counts, tokens=b.tokens, dlogits=dlogits)
    if s["op"] == "combine":
        dy, dw = nv4.moe_combine_backward(s["dout"], s["y"], s["token_row"], s["topk_w"])
        return dict(dy=dy, dtopk_w=dw)
    rule = nv4.NV4_F8_POW2 if s["pow2"] else nv4.NV4_F8_FP32
    f8 = lambda q: nv4.FP8(q["codes"], q["scales"], q["rows"], q["K"], nseg=q["experts"], rule=rule)
    if s["op"] == "quantise":
        if s["layout"] == "rows":
            return nv4.fp8_dequantize(nv4.fp8_quantize(s["x"], rule=rule), torch.float32)
        if s["layout"] == "tiles":
            q = nv4.fp8_quantize(s["x"], layout=nv4.NV4_F8_TILES, nseg=s["experts"], rule=rule)
            return nv4.fp8_dequantize(q, torch.float32)
        seg = dict(nseg=s["experts"], seg_offsets=s["offsets"], seg_padded_offsets=nv4.mx_padded_offsets(s["offsets"]),
                   rule=rule)
        if s["layout"] == "tokens":
            q = nv4.fp8_quantize(s["x"], layout=nv4.NV4_COLS, row_index=s["row_token"], **seg)
            return nv4.fp8_dequantize(q, torch.float32)[:, :s["columns"]]
        q = nv4.fp8_quantize(s["x"], layout=nv4.NV4_ROWS_AND_COLS, **seg)
        return dict(rows=nv4.fp8_dequantize(q.rows_out, torch.float32),
                    tokens=nv4.fp8_dequantize(q, torch.float32)[:, :s["columns"]])
    E, R = s["experts"], s["row_token"].numel()
    if s["form"] == "rows":
        o = dict(M_cap=R, a_rows=s["row_token"] if s["gather"] else None,
                 epilogue=nv4.NV4_EPI_NONE if s["epilogue"] == "none" else nv4.NV4_EPI_SWIGLU)
        if s["epilogue"] == "requantise":
            q = nv4.FP8.empty(R, s["N"], device=s["a"]["codes"].device)
            nv4.fp8_grouped_gemm(f8(s["a"]), f8(s["b"]), s["offsets"], E, s["N"], q_out=q, rule=rule, want_c=False, **o)
            return nv4.fp8_dequantize(q, torch.bfloat16)
        return nv4.fp8_grouped_gemm(f8(s["a"]), f8(s["b"]), s["offsets"], E, s["N"], out_dtype=getattr(torch, s["out"]),
                                    **o)
    padded = nv4.mx_padded_offsets(s["offsets"])
    seg = dict(nseg=E, seg_offsets=s["offsets"], seg_padded_offsets=padded, rule=rule)
    dyc = nv4.fp8_quantize(s["dy"], layout=nv4.NV4_ROWS_AND_COLS, **seg)
    xc = nv4.fp8_quantize(s["x"], layout=nv4.NV4_COLS, row_index=s["row_token"], **seg)
    dx = nv4.fp8_grouped_gemm(dyc.rows_out, f8(s["wt"]), s["offsets"], E, s["K"], M_cap=R, out_dtype=torch.bfloat16)
    dw = nv4.fp8_grouped_gemm(dyc, xc, padded, E, 0, group_mode=nv4.NV4_GROUP_K)
    return dict(dx=dx, dw=dw)


def _values(q, experts=slice(None)):
    """A kept matrix as FP32 values: [rows, K], or [experts, m, K] of these experts' weights."""
    v = q["codes"].view(torch.float8_e4m3fn)
    if not q["experts"]:
        return v.float() * q["scales"].repeat_interleave(BLOCK, 1)[:, :q["K"]]
    v = v.view(q["experts"], -1, q["K"])[experts].float()
    G = q["scales"][experts].repeat_interleave(BLOCK, 2)[:, :, :q["K"]]
    return v * G.repeat_interleave(BLOCK, 1)[:, :v.shape[1]]


def _rounded(x, pow2):
    """The quantised values nearest to x (blocks along the last dimension), FP32."""
    codes, G = _codes(x, pow2)
    return codes.float() * G.repeat_interleave(BLOCK, -1)[..., :x.shape[-1]]


def _by_expert(s, x):
    """Rows in expert order at their padded positions, zeros between: [columns, cols]."""
    out = torch.zeros(s["columns"], x.shape[1], device=DEVICE)
    out[s["slot"]] = x.float()
    return out


def _plain_quantise(s):
    x, pow2 = s["x"].float(), s["pow2"]
    if s["layout"] == "rows":
        return _rounded(x, pow2)
    if s["layout"] == "tiles":
        codes, G = _tiles(x, s["experts"], pow2)
        return _values(_kept(codes, G, s["rows"], s["cols"], s["experts"])).flatten(0, 1)
    if s["layout"] == "tokens":
        return _rounded(_by_expert(s, x[s["row_token"]]).t().contiguous(), pow2)
    return dict(rows=_rounded(x, pow2), tokens=_rounded(_by_expert(s, x).t().contiguous(), pow2))


def _grouped(a, q, sizes):
    """Rows of expert e (sizes[e] of them) times its weights^T: one product per expert with rows."""
    live = [e for e, n in enumerate(sizes) if n]
    b = _values(q, live if len(live) < len(sizes) else slice(None))
    out = torch.empty(a.shape[0], b.shape[1], device=DEVICE)
    at = 0
    for i, e in enumerate(live):
        torch.mm(a[at:at + sizes[e]], b[i].t(), out=out[at:at + sizes[e]])
        at += sizes[e]
    return out


def _plain_product(s):
    E = s["experts"]
    if s["form"] == "rows":
        a = _values(s["a"])
        if s["gather"]:
            a = a[s["row_token"]]
        y = _grouped(a, s["b"], s["sizes"])
        if s["epilogue"] != "none":
            gate, up = y.chunk(2, -1)
            y = gate / (1 + torch.exp(-gate)) * up
        if s["epilogue"] == "requantise":
            y = _rounded(y, s["pow2"])
        return y.to(getattr(torch, s["out"]))
    dx = _grouped(_rounded(s["dy"].float(), s["pow2"]), s["wt"], s["sizes"]).bfloat16()
    dyc = _rounded(_by_expert(s, s["dy"]).t().contiguous(), s["pow2"])
    xc = _rounded(_by_expert(s, s["x"][s["row_token"]]).t().contiguous(), s["pow2"])
    dw = torch.zeros(E, s["N"], s["K"], device=DEVICE)
    at = 0
    for e, n in enumerate(s["sizes"]):
        n = (n + BLOCK - 1) // BLOCK * BLOCK
        torch.mm(dyc[:, at:at + n], xc[:, at:at + n].t(), out=dw[e])
        at += n
    return dict(dx=dx, dw=dw)


def _plain_balance(s):
    T, E, k = s["tokens"], s["experts"], s["k"]
    off = s["seq_offsets"].long()
    nseq = off.numel() - 1
    # the token's sequence: the last one that begins at or before it (empty ones begin there too)
    seq = torch.searchsorted(off[1:], torch.arange(T, device=DEVICE), right=True)
    live = torch.ones(T, device=DEVICE) if s["mask"] is None else s["mask"].float()
    ids = s["topk_ids"].long()
    mx = s["logits"].amax(1, keepdim=True)
    p = torch.exp(s["logits"] - mx)
    total = p.sum(1, keepdim=True)
    p = p / total
    lse = (mx + total.log())[:, 0]
    # sums over each sequence's tokens, in 64 bits: products with the tokens' places
    place = (seq == torch.arange(nseq, device=DEVICE)[:, None]).double() * live.double()
    chosen = torch.zeros(T, E, device=DEVICE, dtype=torch.float64).scatter_add_(1, ids, torch.ones_like(ids).double())
    counts, n = torch.mm(place, chosen), place.sum(1)
    psum, z = torch.mm(place, p.double()), torch.mv(place, lse.double().square())
    div = n.clamp(min=1)
    balance = (E / (k * div * div) * (counts * psum).sum(1)).sum() / nseq
    loss = torch.stack([balance, (z / div).sum() / nseq]).float()
    # gradients
    scale = (E / (nseq * k * div * div)).float()[seq] * live * s["dloss"][0]
    c = counts.float()[seq]
    d = scale[:, None] * p * (c - (c * p).sum(1, keepdim=True))
    d = d + ((2 / (nseq * div)).float()[seq] * live * s["dloss"][1] * lse)[:, None] * p
    chosen, dw = p.gather(1, ids), s["dtopk_w"]
    if s["renorm"]:
        w = chosen / chosen.sum(1, keepdim=True)
        d.scatter_add_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        d -= p * (chosen * dw).sum(1, keepdim=True)
        d.scatter_add_(1, ids, chosen * dw)
    return dict(loss=loss, counts=counts.int(), tokens=n.int(), dlogits=d)


def _plain_combine(s):
    rows = s["token_row"].long().reshape(-1)
    dout = s["dout"].float()
    y = s["y"].float()[rows].view(s["tokens"], s["k"], s["H"])
    dw = (y * dout[:, None]).sum(2)
    dy = torch.empty(rows.numel(), s["H"], device=DEVICE)
    dy[rows] = (s["topk_w"][..., None] * dout[:, None]).flatten(0, 1)
    return dict(dy=dy.to(s["y"].dtype), dtopk_w=dw)


# ------------------------------------------------------------------------------ 64 bits

def _single(x):
    """The FP32 value nearest to a 64-bit one, in 64 bits: the roundings that the format defines."""
    return x.float().double()


def _power(e):
    """2^e in 64 bits from a table (pow and exp2 round)."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=DEVICE)[e.long() + 300]


def _exact_scales(amax, pow2):
    """S of the definition: 448 / amax rounded to FP32, or the power of two at or below it; at most
    2^126, and 1 for a block of zeros."""
    a = torch.where(amax > 0, amax, torch.full_like(amax, 448.0))
    if pow2:
        t = torch.floor(torch.log2(448.0 / a))
        t = torch.where(a * _power(t) > 448.0, t - 1, t)
        t = torch.where(a * _power(t + 1) <= 448.0, t + 1, t)
        return _power(t.clamp(max=126.0))
    return _single(torch.div(torch.full_like(a, 448.0), a).clamp(max=2.0 ** 126))


def _exact_round(x, S):
    """Values of x under scales S (same shape or broadcast): the nearest E4M3 value of fp32(x S),
    halves to even, times fp32(1 / S)."""
    y = _single(x.double() * S)
    m, e = torch.frexp(y.abs())
    step = _power((e - 4).clamp(min=-9))                     # three bits behind the leading one
    q = (torch.round(y.abs() / step) * step).clamp(max=448.0) * torch.sign(y)
    return q * _single(torch.div(torch.ones_like(S), S))


def _exact_rows(x, pow2):
    K = x.shape[-1]
    b = torch.nn.functional.pad(x.double(), (0, -K % BLOCK)).reshape(*x.shape[:-1], -1, BLOCK)
    S = _exact_scales(b.abs().amax(-1, keepdim=True), pow2)
    return _exact_round(b, S).reshape(*x.shape[:-1], -1)[..., :K]


def _exact_tokens(s, x, pow2):
    """[cols, columns]: each expert's rows transposed, its blocks down the tokens."""
    out, lo = torch.zeros(x.shape[1], s["columns"], dtype=torch.float64, device=DEVICE), 0
    for e, n in enumerate(s["sizes"]):
        if n:
            at = int(s["padded"][e])
            out[:, at:at + n] = _exact_rows(x[lo:lo + n].t().double().contiguous(), pow2)
        lo += n
    return out


def _exact_values(q):
    """64-bit values from the bytes: sign, four exponent bits (bias 7), three of significand."""
    c = q["codes"].long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * _power(e - 10), m * 2.0 ** -9)
    v = torch.where(c > 127, -mag, mag)
    row, col = torch.arange(q["rows"], device=DEVICE), torch.arange(q["K"], device=DEVICE) // BLOCK
    if not q["experts"]:
        return v * q["scales"].double()[:, col]
    m = q["rows"] // q["experts"]
    return v * q["scales"].double()[row // m, row % m // BLOCK][:, col]


def _exact_balance(s):
    E, k, off = s["experts"], s["k"], s["seq_offsets"].tolist()
    l, dw = s["logits"].double(), s["dtopk_w"].double()
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    chosen = torch.nn.functional.one_hot(s["topk_ids"].long(), E)            # [T, k, E]
    live = torch.ones_like(lse, dtype=torch.bool) if s["mask"] is None else s["mask"]
    db, dz = s["dloss"].double().tolist()
    w = torch.exp(torch.gather(l, 1, s["topk_ids"].long()) - lse[:, None])
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
        a = w * (dw - (w * dw).sum(1, keepdim=True))
        d = (chosen * a[..., None]).sum(1)
    else:
        d = (chosen * (w * dw)[..., None]).sum(1) - p * (w * dw).sum(1, keepdim=True)
    balance, z, nseq = 0.0, 0.0, len(off) - 1
    for lo, hi in zip(off[:-1], off[1:]):
        at = live[lo:hi].nonzero()[:, 0] + lo
        n = at.numel()
        if n == 0:
            continue
        f = chosen[at].sum((0, 1)).double() * E / (k * n)
        P = p[at]
        balance = balance + (f * P.mean(0)).sum() / nseq
        z = z + lse[at].square().mean() / nseq
        d[at] += db / (nseq * n) * P * (f - (P * f).sum(1, keepdim=True)) + dz * 2 / (nseq * n) * lse[at][:, None] * P
    return dict(loss=torch.tensor([float(balance), float(z)], dtype=torch.float64, device=DEVICE), counts=None, tokens=None,
                dlogits=d)


def exact(case, seed):
    if work(case)["flops"] > MAX_EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s)
    if case["op"] == "combine":
        T, k = case["tokens"], case["k"]
        dout, row = s["dout"].double(), s["token_row"].long()
        dy, dw = torch.zeros(T * k, case["H"], dtype=torch.float64, device=DEVICE), []
        for j in range(k):
            dy[row[:, j]] = s["topk_w"][:, j:j + 1].double() * dout
            dw.append((s["y"][row[:, j]].double() * dout).sum(1))
        return dict(dy=dy, dtopk_w=torch.stack(dw, 1))
    pow2 = case["pow2"]
    if case["op"] == "quantise":
        if case["layout"] == "rows":
            return _exact_rows(s["x"], pow2)
        if case["layout"] == "tokens":
            return _exact_tokens(s, s["x"][s["row_token"].long()], pow2)
        if case["layout"] == "both":
            return dict(rows=_exact_rows(s["x"], pow2), tokens=_exact_tokens(s, s["x"], pow2))
        E, m = case["experts"], case["rows"] // case["experts"]
        out = s["x"].double().view(E, m, case["cols"])
        for r in range(0, m, BLOCK):
            for c in range(0, case["cols"], BLOCK):
                b = out[:, r:r + BLOCK, c:c + BLOCK]
                out[:, r:r + BLOCK, c:c + BLOCK] = _exact_round(b, _exact_scales(b.abs().amax((1, 2), keepdim=True), pow2))
        return out.flatten(0, 1)
    E = case["experts"]
    ends = [sum(s["sizes"][:e]) for e in range(E + 1)]
    if case["form"] == "rows":
        a, b = _exact_values(s["a"]), _exact_values(s["b"]).reshape(E, -1, case["K"])
        if case["gather"]:
            a = a[s["row_token"].long()]
        y = torch.cat([a[ends[e]:ends[e + 1]] @ b[e].t() for e in range(E)])
        if case["epilogue"] != "none":
            N = case["N"]
            y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
        return _exact_rows(y, pow2) if case["epilogue"] == "requantise" else y
    wt = _exact_values(s["wt"]).reshape(E, case["K"], case["N"])
    dy = _exact_rows(s["dy"], pow2)
    dx = torch.cat([dy[ends[e]:ends[e + 1]] @ wt[e].t() for e in range(E)])
    dyc, xc = _exact_tokens(s, s["dy"], pow2), _exact_tokens(s, s["x"][s["row_token"].long()], pow2)
    pad = s["padded"].tolist()
    dw = torch.stack([dyc[:, pad[e]:pad[e + 1]] @ xc[:, pad[e]:pad[e + 1]].t() for e in range(E)])
    return dict(dx=dx, dw=dw)


# ------------------------------------------------------------------------------ floors

def _f8_bytes(rows, K):
    return rows * (K + 4 * ((K + BLOCK - 1) // BLOCK))


def _experts_read(tokens, k, experts):
    """Experts that some token chooses, on average over even routing."""
    return experts * (1 - (1 - k / experts) ** tokens)


def work(case):
    size = {BF16: 2, FP32: 4}
    if case["op"] == "quantise":
        n, layout = case["rows"] * case["cols"], case["layout"]
        out = n * case["k"] if layout == "tokens" else 2 * n if layout == "both" else n
        index = 4 * case["rows"] * case["k"] if layout == "tokens" else 0
        return dict(bytes=n * size[case["dtype"]] + 4 * out + index, flops=4 * out)
    T, k = case["tokens"], case["k"]
    R = T * k
    if case["op"] == "combine":
        H = case["H"]
        return dict(bytes=T * H * size[case["out"]] + 2 * R * H * size[case["rows"]] + 12 * R, flops=3 * R * H)
    E = case["experts"]
    if case["op"] == "balance":
        return dict(bytes=8 * T * E + 8 * R + 4 * case["sequences"] * E, flops=12 * T * E)
    K, N = case["K"], case["N"]
    read = _experts_read(T, k, E)
    if case["form"] == "gradients":
        return dict(bytes=2 * R * N + 2 * T * K + 4 * R + int(read * N * K) + 2 * R * K + 4 * E * N * K,
                    flops=4 * R * N * K)
    n = N * (1 if case["epilogue"] == "none" else 2)
    a = _f8_bytes(T, K) + 4 * R if case["gather"] else _f8_bytes(R, K)
    return dict(bytes=a + int(read * n * K) + R * N * size[case["out"]], flops=2 * R * n * K)
