"""The bf16 GroupedLinear gradients and the adapter linear as they are measured: cases,
inputs, plain forms.

Two kinds of case:
  bwd    the backward pass of a bf16 GroupedLinear: the gradients of its input, of every
         expert's weights (bf16, or fp32 as an optimizer's gradient buffer holds them) and
         of the row scales, if it has any.
  lora   a projection shared by many requests, with the low-rank adapter of each request
         beside it: y = x w^T + s (x a^T) b^T with every row's own a, b and s.
"""
import math

import torch

own = False

DEV = "cuda:0"


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # a layer small enough for latency to count: 256 tokens on 2 of 4 experts
        {"name": "bwd 4 small experts", "op": "bwd", "M": 512, "E": 4, "K": 128, "N": 256,
         "loads": "even", "scaled": False, "dw": "bf16"},
        # a short sample on 8 large experts: reading the weights and writing their gradients
        {"name": "bwd short sample", "op": "bwd", "M": 64, "E": 8, "K": 4096, "N": 14336,
         "loads": "zipf", "scaled": False, "dw": "bf16"},
        # 8192 tokens on 2 of 8 middle-sized experts, routing weights applied to the output
        {"name": "bwd 8 experts scaled", "op": "bwd", "M": 16384, "E": 8, "K": 1024, "N": 2816,
         "loads": "zipf", "scaled": True, "dw": "bf16"},
        # odd counts and a last tile of each kind
        {"name": "bwd odd sizes", "op": "bwd", "M": 1003, "E": 7, "K": 1408, "N": 2064,
         "loads": "zipf", "scaled": True, "dw": "bf16"},
        # 64 fine-grained experts, every eighth idle, gradients kept in fp32
        {"name": "bwd 64 experts fp32", "op": "bwd", "M": 65536, "E": 64, "K": 2048, "N": 2816,
         "loads": "gaps", "scaled": False, "dw": "fp32"},
        # the down projection of 16384 tokens on 2 of 8 large experts, unevenly loaded
        {"name": "bwd down projection", "op": "bwd", "M": 32768, "E": 8, "K": 14336, "N": 4096,
         "loads": "zipf", "scaled": True, "dw": "bf16"},
        # one sequence decoding with its adapter
        {"name": "lora one token", "op": "lora", "M": 1, "K": 4096, "N": 4096, "r": 16, "L": 8,
         "none": 0.0, "batch": "tokens"},
        # sixteen sequences decoding, each with one of 32 adapters
        {"name": "lora 16 tokens", "op": "lora", "M": 16, "K": 4096, "N": 14336, "r": 64, "L": 32,
         "none": 0.1, "batch": "tokens"},
        # a hundred sequences on a narrow projection, a third of them without an adapter
        {"name": "lora 100 tokens", "op": "lora", "M": 100, "K": 2048, "N": 2816, "r": 8, "L": 64,
         "none": 0.33, "batch": "tokens"},
        # a chunk of prompts among decoding sequences
        {"name": "lora mixed batch", "op": "lora", "M": 1003, "K": 4096, "N": 4096, "r": 32,
         "L": 16, "none": 0.1, "batch": "mixed"},
        # odd sizes, a rank that is no power of two
        {"name": "lora odd sizes", "op": "lora", "M": 5001, "K": 1408, "N": 2064, "r": 24, "L": 5,
         "none": 0.2, "batch": "prompts"},
        # prompts of several requests on a large layer's up projection
        {"name": "lora prompts", "op": "lora", "M": 16384, "K": 4096, "N": 14336, "r": 16, "L": 8,
         "none": 0.1, "batch": "prompts"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        E = _log_int(rng, 1, 64)
        loads = rng.choice(["even", "zipf", "gaps"])
        M = _log_int(rng, 1, 32768)
        K, N = 32 * _log_int(rng, 1, 448), 16 * _log_int(rng, 1, 896)
        while E * K * N > 1 << 29:
            E = max(1, E // 2)
        while M * K * N > 1 << 40:
            M //= 2
        scaled = rng.random() < 0.5
        return {"op": "bwd", "M": M, "E": E, "K": K, "N": N, "loads": loads, "scaled": scaled,
                "dw": "bf16" if scaled else rng.choice(["bf16", "fp32"])}
    M = _log_int(rng, 1, 16384)
    K, N = 32 * _log_int(rng, 1, 224), 16 * _log_int(rng, 1, 896)
    while M * K * N > 1 << 39:
        M //= 2
    return {"op": "lora", "M": M, "K": K, "N": N, "r": rng.choice([8, 16, 16, 24, 32, 64, 128]),
            "L": _log_int(rng, 1, 64), "none": rng.choice([0.0, 0.1, 0.5]),
            "batch": rng.choice(["tokens", "mixed", "prompts"])}


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


def _requests(case):
    """Rows of each request: one (tokens), about a seventh of the batch (prompts), or half
    the batch in three prompts and the rest one each (mixed)."""
    M = case["M"]
    if case["batch"] == "tokens":
        return [1] * M
    if case["batch"] == "prompts":
        n = max(1, M // 7)
        return [n] * (M // n) + ([M % n] if M % n else [])
    n = M // 6
    return [n] * 3 * (n > 0) + [1] * (M - 3 * n)


# ---- inputs ---------------------------------------------------------------------

def _acts(g, shape):
    """Activations: unit normal with one value in a hundred twenty times as large."""
    x = torch.randn(shape, generator=g, device=DEV)
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.01, 20 * x, x).bfloat16()


def _normal(g, shape, scale):
    return (torch.randn(shape, generator=g, device=DEV) * scale).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "bwd":
        E, counts = case["E"], _counts(case)
        off = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(DEV)
        w = torch.stack([_normal(g, (N, K), 0.02) for _ in range(E)])
        return {"op": "bwd", "dy": _normal(g, (M, N), 1.0), "x": _acts(g, (M, K)), "offsets": off,
                "most": max(counts), "w": w, "dw": case["dw"],
                "r": torch.rand(M, generator=g, device=DEV) if case["scaled"] else None}
    L, r, lengths = case["L"], case["r"], _requests(case)
    pick = torch.randint(0, L, (len(lengths),), generator=g, device=DEV)
    bare = torch.rand(len(lengths), generator=g, device=DEV) < case["none"]
    ids = torch.where(bare, -1, pick).repeat_interleave(torch.tensor(lengths, device=DEV))
    return {"op": "lora", "x": _acts(g, (M, K)), "w": _normal(g, (N, K), 0.02),
            "a": _normal(g, (L, r, K), K ** -0.5), "b": _normal(g, (L, N, r), 0.02),
            "ids": ids.int().contiguous(),
            "scale": 0.5 + 1.5 * torch.rand(L, generator=g, device=DEV)}


# ---- one pass -------------------------------------------------------------------

def _run_own(s):
    import grouped_gemm_mxfp8_amd as gm
    if s["op"] == "lora":
        return gm.lora_linear_fwd(s["x"], s["w"], s["a"], s["b"], s["ids"], scale=s["scale"])
    dtype = torch.float32 if s["dw"] == "fp32" else torch.bfloat16
    dx, dw, dr = gm.grouped_linear_bwd(s["dy"], s["x"], s["offsets"], s["w"], row_scale=s["r"],
                                       dw_dtype=dtype)
    return (dx, dw) if dr is None else (dx, dw, dr)


def _plain_bwd(s):
    dy, x, w, off, most = s["dy"].float(), s["x"].float(), s["w"].float(), s["offsets"], s["most"]
    E, N, K = w.shape
    # every expert's rows in a slab of as many rows as the fullest one has
    row = torch.arange(x.shape[0], device=x.device)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    at = e * most + (row - off[e])
    dys, xs = (torch.zeros((E * most, t.shape[1]), device=x.device) for t in (dy, x))
    dys[at], xs[at] = dy, x
    g = torch.bmm(dys.view(E, most, N), w).view(E * most, K)[at]
    dr = None
    if s["r"] is not None:
        dr = (g * x).sum(1)
        g = g * s["r"][:, None]
        dys[at] = dy * s["r"][:, None]
    dw = torch.bmm(dys.view(E, most, N).transpose(1, 2), xs.view(E, most, K))
    dw = dw if s["dw"] == "fp32" else dw.bfloat16()
    return (g.bfloat16(), dw) if dr is None else (g.bfloat16(), dw, dr)


def _plain_lora(s):
    x, ids = s["x"].float(), s["ids"]
    L, r, K = s["a"].shape
    # every adapter on every row, then only the row's own
    h = (x @ s["a"].float().view(L * r, K).t()).view(-1, L, r)
    mine = ids[:, None] == torch.arange(L, device=x.device)
    h = torch.where(mine[..., None], h * s["scale"][:, None], 0.0)
    b = s["b"].float().transpose(1, 2).reshape(L * r, -1)
    return (x @ s["w"].float().t() + h.view(-1, L * r) @ b).bfloat16()


def run(state):
    if own:
        return _run_own(state)
    return _plain_bwd(state) if state["op"] == "bwd" else _plain_lora(state)


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "bwd":
        used = sum(c > 0 for c in _counts(case))
        grad = 4 if case["dw"] == "fp32" else 2
        return {"bytes": 2 * M * (N + K) + 2 * used * N * K + 2 * M * K + grad * case["E"] * N * K
                + (8 * M if case["scaled"] else 0), "flops": 4 * M * N * K}
    L, r, lengths = case["L"], case["r"], _requests(case)
    share = 1 - case["none"]                  # of the requests, on average
    used = L * (1 - (1 - share / L) ** len(lengths))
    return {"bytes": 2 * M * K + 2 * N * K + 2 * used * r * (K + N) + 2 * M * N + 4 * M,
            "flops": 2 * M * N * K + 2 * share * M * r * (K + N)}


# ---- the definition in 64 bits -----------------------------------------------------

def _exact_bwd(case, s):
    at = s["offsets"].tolist()
    dx, dw, dr = [], [], []
    for e in range(case["E"]):
        rows = slice(at[e], at[e + 1])
        dy, x, w = s["dy"][rows].double(), s["x"][rows].double(), s["w"][e].double()
        r = None if s["r"] is None else s["r"][rows].double()
        scaled = dy if r is None else torch.mul(dy, r.unsqueeze(1))
        dx.append(torch.matmul(scaled, w))
        dw.append(torch.matmul(scaled.t(), x))
        if r is not None:                     # the output row without its scale, against dy
            dr.append(torch.mul(torch.matmul(x, w.t()), dy).sum(dim=1))
    out = (torch.cat(dx), torch.stack(dw))
    return out if s["r"] is None else (*out, torch.cat(dr))


def _exact_lora(case, s):
    x, ids = s["x"].double(), s["ids"].long()
    y = torch.matmul(x, s["w"].double().t())
    for i in range(case["L"]):
        rows = torch.nonzero(ids == i).flatten()
        low = torch.matmul(x[rows], s["a"][i].double().t())
        y[rows] += s["scale"][i].double() * torch.matmul(low, s["b"][i].double().t())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_bwd(case, s) if case["op"] == "bwd" else _exact_lora(case, s)
