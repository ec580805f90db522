"""The MXFP4 and few-token operators as they are measured: cases, inputs, plain forms.

Three kinds of case:
  quantize  bf16 -> MXFP4 codes and scales -> the bf16 values they stand for
            (rowwise, or the columnwise copy of a batch of matrices).
  linear    GroupedLinear on MXFP4 weights: the activations are quantized (to
            MXFP4 or MXFP8) and multiplied with their expert's weights.
  layer     a whole MoE layer for a few tokens: routing, gate-up, SwiGLU,
            down projection and combine, on bf16, MXFP8 or MXFP4 weights.
"""
import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decoded token's activations: latency
        {"name": "quantize one token", "op": "quantize", "axis": "row", "B": 1, "R": 1, "C": 4096},
        # a prompt's activations, hidden size 4096
        {"name": "quantize prompt", "op": "quantize", "axis": "row", "B": 1, "R": 16384, "C": 4096},
        # a ragged batch over a fine-grained expert's inner size
        {"name": "quantize odd rows", "op": "quantize", "axis": "row", "B": 1, "R": 1003, "C": 1408},
        # 64 experts' down projections, laid out for the data gradient
        {"name": "quantize 64 experts by columns", "op": "quantize", "axis": "col", "B": 64,
         "R": 2048, "C": 1408},
        # gate-up projection of a prompt, 8 experts evenly loaded, both sides 4 bits
        {"name": "linear fp4 prompt", "op": "linear", "x": "mxfp4", "M": 16384, "E": 8, "K": 4096,
         "N": 28672, "loads": "even", "scaled": False},
        # down projection of a batch with uneven expert loads, routing weights applied
        {"name": "linear fp8 x fp4 zipf", "op": "linear", "x": "mxfp8", "M": 32768, "E": 8,
         "K": 14336, "N": 4096, "loads": "zipf", "scaled": True},
        # 64 small experts, every eighth idle, about 140 rows each
        {"name": "linear fp8 x fp4 64 experts", "op": "linear", "x": "mxfp8", "M": 8023, "E": 64,
         "K": 2048, "N": 2816, "loads": "gaps", "scaled": True},
        # sixteen rows in flight over 8 experts: the weights are what is read
        {"name": "linear fp4 decode", "op": "linear", "x": "mxfp4", "M": 16, "E": 8, "K": 4096,
         "N": 28672, "loads": "zipf", "scaled": False},
        # one sequence decoding on 8 large experts with 4-bit weights
        {"name": "layer fp4 one token", "op": "layer", "w": "mxfp4", "T": 1, "pad": 0, "E": 8,
         "k": 2, "H": 4096, "F": 14336},
        # sixteen sequences decoding on the same experts, unquantized
        {"name": "layer bf16 16 tokens", "op": "layer", "w": "bf16", "T": 16, "pad": 0, "E": 8,
         "k": 2, "H": 4096, "F": 14336},
        # 64 sequences on 64 fine-grained experts
        {"name": "layer fp4 64 tokens", "op": "layer", "w": "mxfp4", "T": 64, "pad": 0, "E": 64,
         "k": 8, "H": 2048, "F": 1408},
        # five sequences in a batch padded to eight (padding rows mask every expert)
        {"name": "layer fp8 padded batch", "op": "layer", "w": "mxfp8", "T": 8, "pad": 3, "E": 64,
         "k": 8, "H": 2048, "F": 1408},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "layer", "layer"])
    if op == "quantize":
        if rng.random() < 0.6:
            return {"op": op, "axis": "row", "B": 1, "R": _log_int(rng, 1, 16384),
                    "C": BLOCK * _log_int(rng, 1, 128)}
        return {"op": op, "axis": "col", "B": _log_int(rng, 1, 32),
                "R": BLOCK * _log_int(rng, 1, 64), "C": BLOCK * _log_int(rng, 1, 64)}
    if op == "linear":
        E = _log_int(rng, 1, 64)
        K, N = BLOCK * _log_int(rng, 1, 256), BLOCK * _log_int(rng, 2, 256)
        while E * K * N > 1 << 30:
            E = max(1, E // 2)
        return {"op": op, "x": rng.choice(["mxfp4", "mxfp8"]), "M": _log_int(rng, 1, 16384), "E": E,
                "K": K, "N": N, "loads": rng.choice(["even", "zipf", "gaps"]),
                "scaled": rng.random() < 0.5}
    E = _log_int(rng, 2, 128)
    H, F = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 64)
    while E * H * F > 3 << 28:
        E = max(2, E // 2)
    T = _log_int(rng, 1, 128)
    return {"op": op, "w": rng.choice(["bf16", "mxfp8", "mxfp4"]), "T": T,
            "pad": rng.choice([0, 0, T // 3]), "E": E, "k": rng.randint(1, min(E, 8)), "H": H,
            "F": F}


def _counts(case):
    """Rows of each expert: even, falling as 1 / rank^1.1, or even with every
    eighth expert idle (the last one of each eight)."""
    M, E = case["M"], case["E"]
    if case["loads"] == "zipf":
        share = [(e + 1) ** -1.1 for e in range(E)]
    elif case["loads"] == "gaps":
        share = [0.0 if e % 8 == 7 else 1.0 for e in range(E)]
    else:
        share = [1.0] * E
    total, done, run, counts = sum(share), 0, 0.0, []
    for s in share:
        run += s
        upto = min(M, int(M * run / total + 0.5))
        counts.append(upto - done)
        done = upto
    counts[0] += M - done
    return counts


# ---- formats (plain torch) -----------------------------------------------------

def _exponent(v):
    """floor(log2 v) of positive v (0 gives a very small number)."""
    return torch.where(v > 0, torch.frexp(v)[1] - 1, torch.full_like(v, -10000, dtype=torch.int32))


def _pow2(e, dtype):
    """2^e, -149 <= e <= 127, exactly (the device's pow and ldexp are not exact)."""
    bits = torch.where(e >= -126, (e + 127) << 23, 1 << (e + 149).clamp(min=0, max=22))
    return bits.int().view(torch.float32).to(dtype)


def _round_e2m1(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(v.dtype)
    return torch.copysign(torch.round(a / step) * step, v)


def _round_e4m3(v):
    a = v.abs().clamp(max=448.0)
    step = _pow2(_exponent(a).clamp(min=-6) - 3, v.dtype)
    return torch.copysign(torch.round(a / step) * step, v)


def _blocks(x, fmt):
    """(rounded values of the scaled elements [..., C/32, 32], block exponents [..., C/32])."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = 2 if fmt == "mxfp4" else 8
    X = (_exponent(b.abs().amax(-1)) - top).clamp(min=-127)
    v = b / _pow2(X, b.dtype)[..., None]
    return (_round_e2m1(v) if fmt == "mxfp4" else _round_e4m3(v)), X


def _fake(x, fmt):
    """The values that the block-quantized x stands for."""
    q, X = _blocks(x, fmt)
    return (q * _pow2(X, q.dtype)[..., None]).flatten(-2)


def _encode(x, fmt):
    """Codes (two 4-bit codes a byte, the even element low) and scales of x."""
    q, X = _blocks(x.float(), fmt)
    q = q.flatten(-2)
    if fmt == "mxfp4":
        a = q.abs()
        c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
        c |= torch.signbit(q).to(torch.uint8) << 3
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    else:
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.contiguous(), (X + 127).to(torch.uint8)


def _decode(w, dtype):
    """Values of weights as prepare() lays them out: a bf16 tensor or (codes, scales, format)."""
    if isinstance(w, torch.Tensor):
        return w.to(dtype)
    codes, scales, fmt = w
    if fmt == "mxfp4":
        t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
        i = torch.arange(256, device=codes.device)
        v = torch.stack([t[i & 15], t[i >> 4]], -1)[codes.int()].flatten(-2)
    else:
        v = codes.view(torch.float8_e4m3fn).to(dtype)
    s = _pow2(scales.int() - 127, dtype)
    return (v.unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def _select(w, e):
    return w[e] if isinstance(w, torch.Tensor) else (w[0][e], w[1][e], w[2])


# ---- inputs ---------------------------------------------------------------------

def _acts(g, shape):
    """Activations: unit normal with one value in a hundred twenty times as large."""
    x = torch.randn(shape, generator=g, device=DEV)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.01, 20 * x, x).bfloat16()


def _weights(g, E, N, K, fmt):
    parts = [(torch.randn((N, K), generator=g, device=DEV) * 0.02).bfloat16() for _ in range(E)]
    if fmt == "bf16":
        return torch.stack(parts)
    enc = [_encode(p, fmt) for p in parts]
    return torch.stack([c for c, _ in enc]), torch.stack([s for _, s in enc]), fmt


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "quantize":
        B, R, C = case["B"], case["R"], case["C"]
        x = _acts(g, (R, C) if B == 1 else (B, R, C))
        return {"op": "quantize", "axis": case["axis"], "x": x}
    if case["op"] == "linear":
        counts = _counts(case)
        off = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(DEV)
        return {"op": "linear", "fmt": case["x"], "x": _acts(g, (case["M"], case["K"])),
                "offsets": off, "most": max(counts),
                "w": _weights(g, case["E"], case["N"], case["K"], "mxfp4"),
                "r": torch.rand(case["M"], generator=g, device=DEV) if case["scaled"] else None}
    T, E, H, F = case["T"], case["E"], case["H"], case["F"]
    logits = torch.randn((T, E), generator=g, device=DEV)
    if case["pad"]:
        logits[T - case["pad"]:] = -math.inf
    return {"op": "layer", "fmt": case["w"], "x": _acts(g, (T, H)), "logits": logits,
            "k": case["k"], "w1": _weights(g, E, 2 * F, H, case["w"]),
            "w2": _weights(g, E, H, F, case["w"])}


# ---- one pass -------------------------------------------------------------------

def _own_weights(gm, w):
    if isinstance(w, torch.Tensor):
        return w
    return (gm.Mx4Tensor if w[2] == "mxfp4" else gm.MxTensor)(w[0], w[1])


def _run_own(s):
    import grouped_gemm_mxfp8_amd as gm
    if s["op"] == "quantize":
        row = s["axis"] == "row"
        q = gm.mxfp4_quantize(s["x"], rowwise=row, colwise=not row)
        return gm.mxfp4_dequantize(q[s["axis"]])
    if s["op"] == "linear":
        quantize = gm.mxfp4_quantize if s["fmt"] == "mxfp4" else gm.mxfp8_quantize
        return gm.grouped_linear_fwd(quantize(s["x"])["row"], s["offsets"],
                                     _own_weights(gm, s["w"]), row_scale=s["r"])
    return gm.moe_layer_fwd(s["x"], s["logits"], _own_weights(gm, s["w1"]),
                            _own_weights(gm, s["w2"]), s["k"])


def _plain_quantize(s):
    x = s["x"].float()
    if s["axis"] == "col":
        x = x.transpose(-1, -2).contiguous()
    return _fake(x, "mxfp4").bfloat16()


def _plain_linear(s):
    x, off, most = _fake(s["x"].float(), s["fmt"]), s["offsets"], s["most"]
    w = _decode(s["w"], torch.float32)
    E, N, K = w.shape
    # every expert's rows in a slab of as many rows as the fullest one has
    row = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = e * most + (row - off[e])
    slabs = torch.zeros((E * most, K), device=x.device)
    slabs[at] = x
    y = torch.bmm(slabs.view(E, most, K), w.transpose(1, 2)).view(E * most, N)[at]
    if s["r"] is not None:
        y = y * s["r"][:, None]
    return y.bfloat16()


def _top_k(logits, k):
    """The k largest logits of every row (the lower expert among equal ones) and the softmax
    of them; a row of -inf alone has no experts (weights 0)."""
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    m = torch.where(torch.isinf(v[:, :1]), 0.0, v[:, :1])
    p = torch.exp(v - m)
    n = p.sum(1, keepdim=True)
    return ids, torch.where(n > 0, p / n, 0.0)


def _plain_layer(s):
    x, k, w1, w2 = s["x"].float(), s["k"], s["w1"], s["w2"]
    ids, r = _top_k(s["logits"], k)
    T, E = s["logits"].shape
    mx = s["fmt"] != "bf16"
    if mx:
        x = _fake(x, "mxfp8")
    if T * k <= E:        # the slots' own weights, one copy a slot
        pick = ids.flatten()
        w1, w2 = _select(w1, pick), _select(w2, pick)
        xs, rs = x.repeat_interleave(k, 0)[:, None], r.flatten()[:, None, None]
    else:                 # every expert on every token
        xs = x.expand(E, -1, -1)
        rs = torch.zeros((T, E), device=x.device).scatter(1, ids, r).t()[..., None]
    h = torch.bmm(xs, _decode(w1, torch.float32).transpose(1, 2))
    a, b = h.chunk(2, -1)
    z = rs * (a / (1 + torch.exp(-a)) * b)
    z = _fake(z, "mxfp8") if mx else z.bfloat16().float()
    y = torch.bmm(z, _decode(w2, torch.float32).transpose(1, 2))
    y = y.view(T, k, -1).sum(1) if T * k <= E else y.sum(0)
    return y.bfloat16()


def run(state):
    if own:
        return _run_own(state)
    return {"quantize": _plain_quantize, "linear": _plain_linear,
            "layer": _plain_layer}[state["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------

_PER_VALUE = {"bf16": 2.0, "mxfp8": 33 / 32, "mxfp4": 17 / 32}


def work(case):
    if case["op"] == "quantize":
        n = case["B"] * case["R"] * case["C"]
        return {"bytes": n * (2 + 2 * _PER_VALUE["mxfp4"] + 2), "flops": 0}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        used = sum(c > 0 for c in _counts(case))
        return {"bytes": 2 * M * K + used * N * K * _PER_VALUE["mxfp4"] + 2 * M * N
                + (4 * M if case["scaled"] else 0), "flops": 2 * M * N * K}
    T, E, k, H, F = (case[n] for n in ("T", "E", "k", "H", "F"))
    live = T - case["pad"]
    used = E * (1 - (1 - k / E) ** live)      # experts that some token picks, on average
    return {"bytes": used * 3 * H * F * _PER_VALUE[case["w"]] + 4 * T * H + 4 * T * E,
            "flops": 6 * live * k * H * F}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_two(e):
    """2^e of whole e in [-160, 160] (float64), from a table: the device's pow is not exact."""
    table = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=DEV)
    return table[e.long() + 160]


def _exact_block(x, levels, top):
    """Block quantization by its definition: the scale is the largest power of two at which
    the block's amax falls under 2^(top + 1), and each element goes to the nearest level
    (the even one of two equally near, saturating)."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().max(-1).values
    X = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    X = torch.where(_exact_two(X) > amax, X - 1, X)         # log2 may be off either way
    X = torch.where(_exact_two(X + 1) <= amax, X + 1, X)
    X = torch.where(amax > 0, (X - top).clamp(min=-127), torch.full_like(X, -127.0))
    s = _exact_two(X)[..., None]
    a = (b / s).abs().clamp(max=levels[-1].item())
    hi = torch.searchsorted(levels, a).clamp(max=len(levels) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - levels[lo], levels[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    q = torch.where(up, levels[hi], levels[lo])
    return (torch.copysign(q, b) * s).reshape(x.shape)


def _levels(fmt):
    if fmt == "mxfp4":
        v = list(E2M1)
    else:
        v = [m * 2.0 ** -9 for m in range(8)]
        v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device=DEV), (2 if fmt == "mxfp4" else 8)


def _exact_quant(x, fmt):
    lv, top = _levels(fmt)
    return _exact_block(x, lv, top)


def _exact_weights(w, e):
    if isinstance(w, torch.Tensor):
        return w[e].double()
    codes, scales, fmt = w[0][e].long(), w[1][e], w[2]
    lv, _ = _levels(fmt)
    if fmt == "mxfp4":
        codes = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
        v, neg = lv[codes & 7], codes & 8
    else:
        v, neg = lv[codes & 127], codes & 128
    s = _exact_two(scales.long() - 127).repeat_interleave(BLOCK, -1)
    return torch.where(neg > 0, -v, v) * s


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        x = s["x"]
        rows = (x if s["axis"] == "row" else x.mT).reshape(-1, x.shape[-1 if s["axis"] == "row" else -2])
        out = torch.cat([_exact_quant(part.double(), "mxfp4") for part in rows.split(1 << 14)])
        return out.reshape(x.shape if s["axis"] == "row" else x.mT.shape)
    if s["op"] == "linear":
        out, at = [], s["offsets"].tolist()
        for e in range(case["E"]):
            if at[e + 1] > at[e]:
                w = _exact_weights(s["w"], e)
                for part in s["x"][at[e]:at[e + 1]].split(2048):
                    out.append(_exact_quant(part.double(), s["fmt"]) @ w.t())
        y = torch.cat(out)
        return y if s["r"] is None else y * s["r"].double()[:, None]
    T, E, k = case["T"], case["E"], case["k"]
    logits = s["logits"].double().cpu()
    order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    r = torch.zeros((T, E), dtype=torch.float64)
    for t in range(T - case["pad"]):
        v = logits[t, order[t]]
        r[t, order[t]] = torch.softmax(v, 0)
    r = r.to(DEV)
    x = s["x"].double()
    if s["fmt"] != "bf16":
        x = _exact_quant(x, "mxfp8")
    y = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
    for e in range(E):
        rows = torch.nonzero(r[:, e] > 0).flatten()
        if len(rows):
            h = x[rows] @ _exact_weights(s["w1"], e).t()
            a, b = h[:, :case["F"]], h[:, case["F"]:]
            z = r[rows, e, None] * a * torch.sigmoid(a) * b
            z = _exact_quant(z, "mxfp8") if s["fmt"] != "bf16" else z.bfloat16().double()
            y[rows] += z @ _exact_weights(s["w2"], e).t()
    return y
