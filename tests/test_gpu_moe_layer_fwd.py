"""The whole MoE layer for a few tokens on the GPU against the FP64 oracle.

Bounds.  The output has one bf16 rounding: 2^-8 of each value, about 1.7e-3 in
Frobenius norm.  z is rounded to E4M3 blocks (or bf16) from fp32 sums that
differ from the oracle's by some 1e-6, so a few of the F z values of a row may
round to the neighbouring code, off by at most 2^-3 (bf16: 2^-7) of
themselves: one such value changes an output by 2^-3 |z w2|, which against the
row's RMS of sqrt(F) |z w2| is 2^-3 / sqrt(F) times a few for the largest
product (1.1e-2 times a few at F = 128, the smallest used).  The repository's
parity bar for fused outputs, 1e-2 in norm and 5e-2 of a row's RMS, covers
both; for bf16 weights the neighbour is 16 times nearer, and 4e-3 and 3e-2 (the
bar for products of the same codes) are used."""
import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import mx4_oracle as P
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu
FMTS = ["bf16", "mxfp8", "mxfp4"]


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


def quant(w, fmt):
    if fmt == "bf16":
        return w
    return (gm.mxfp4_quantize if fmt == "mxfp4" else gm.mxfp8_quantize)(w)["row"]


def values(w):
    if isinstance(w, torch.Tensor):
        return to64(w)
    c, s = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    return P.dequantize4_lastdim(c, s) if isinstance(w, gm.Mx4Tensor) else O.dequantize_lastdim(c, s)


def make(T, E, H, F, fmt, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    x = rand(T, H).bfloat16()
    w1 = quant((rand(E, 2 * F, H) * H ** -0.5).bfloat16(), fmt)
    w2 = quant((rand(E, H, F) * F ** -0.5).bfloat16(), fmt)
    return x, rand(T, E), w1, w2


def check(out, x, logits, w1, w2, k, fmt):
    ref = P.moe_layer(to64(x), to64(logits), values(w1), values(w2), k, fmt != "bf16")
    got = to64(out)
    assert np.isfinite(got).all()
    zero = ~ref.any(axis=1)
    assert not got[zero].any()
    if zero.all():
        return
    rel, row = O.parity_metrics(got[~zero], ref[~zero])
    bar = (4e-3, 3e-2) if fmt == "bf16" else (1e-2, 5e-2)
    assert rel <= bar[0] and row <= bar[1], (rel, row)


SHAPES = [  # T, E, k, H, F
    (1, 1, 1, 128, 128),
    (1, 8, 2, 256, 384),
    (1, 64, 8, 512, 1408),        # F = 11 steps of 128
    (2, 4, 4, 128, 256),          # every expert on every token
    (5, 16, 3, 384, 128),
    (16, 8, 2, 512, 512),
    (17, 8, 2, 256, 256),         # one token over a column tile
    (31, 2, 1, 256, 640),
    (33, 3, 2, 128, 256),
    (64, 64, 8, 256, 384),
    (100, 2, 2, 256, 256),        # 100 rows an expert: more than one chunk
    (128, 4, 1, 384, 256),
    (128, 70, 5, 128, 128),       # more than 64 experts
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,k,H,F", SHAPES)
def test_against_the_oracle(dev, T, E, k, H, F, fmt):
    x, logits, w1, w2 = make(T, E, H, F, fmt, T * E + F, dev)
    out = gm.moe_layer_fwd(x, logits, w1, w2, k)
    torch.cuda.synchronize()
    check(out, x, logits, w1, w2, k, fmt)
    assert torch.equal(out, gm.moe_layer_fwd(x, logits, w1, w2, k))


@pytest.mark.parametrize("T,fmt", [(3, "mxfp4"), (40, "mxfp8"), (128, "bf16"), (128, "mxfp4")])
def test_1024_experts_64_slots(dev, T, fmt):
    """The largest plan (8192 rows at T = 128)."""
    x, logits, w1, w2 = make(T, 1024, 128, 128, fmt, 5, dev)
    out = gm.moe_layer_fwd(x, logits, w1, w2, 64)
    torch.cuda.synchronize()
    check(out, x, logits, w1, w2, 64, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,k,H,F", [
    (1, 2, 1, 4096, 14336),
    (20, 3, 2, 7168, 2048),
    (48, 5, 2, 2816, 1920),
])
def test_real_sizes_against_the_oracle(dev, T, E, k, H, F, fmt):
    x, logits, w1, w2 = make(T, E, H, F, fmt, H + F, dev)
    out = gm.moe_layer_fwd(x, logits, w1, w2, k)
    torch.cuda.synchronize()
    check(out, x, logits, w1, w2, k, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("F", [384, 512])
@pytest.mark.parametrize("E", [64, 512])
def test_large_plans_with_many_rows_an_expert(dev, E, F, fmt):
    """128 tokens, 64 slots: the plan leaves the LDS of a down workgroup to one
    tile of W2, with two (512 experts) or four (64) tiles of rows; F of whole
    and of partial groups of steps."""
    x, logits, w1, w2 = make(128, E, 128, F, fmt, E + F, dev)
    out = gm.moe_layer_fwd(x, logits, w1, w2, 64)
    torch.cuda.synchronize()
    check(out, x, logits, w1, w2, 64, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,k", [(60, 64, 4), (100, 32, 2), (128, 128, 8)])
def test_all_tokens_on_the_same_experts(dev, T, E, k, fmt):
    """Far more rows on an expert than the even spread that the row tiles are
    chosen for: its rows come in several turns."""
    x, logits, w1, w2 = make(T, E, 256, 384, fmt, T + E, dev)
    logits[:, 5:5 + k] += 50.0
    out = gm.moe_layer_fwd(x, logits, w1, w2, k)
    torch.cuda.synchronize()
    check(out, x, logits, w1, w2, k, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_masked_experts_ties_and_padding_rows(dev, fmt):
    T, E, k = 9, 8, 3
    x, logits, w1, w2 = make(T, E, 256, 256, fmt, 3, dev)
    inf = float("inf")
    logits[0] = 1.5                                   # ties: experts 0, 1, 2
    logits[1] = -inf                                  # a padding row
    logits[2] = -inf
    logits[2, 6] = 0.25                               # one expert left of three slots
    logits[3, :5] = -inf
    logits[4] = torch.finfo(torch.float32).min        # the type's lowest value is a value
    logits[5, 2] = float("nan")                       # masked
    logits[6] = torch.tensor([0.0, -0.0, 0.0, -1, -1, -1, -0.0, 2.0], device=dev)
    logits[8] = -inf
    x[8] = inf                                        # a padding row's contents do not matter
    out = gm.moe_layer_fwd(x, logits, w1, w2, k)
    torch.cuda.synchronize()
    assert not out[1].any() and not out[8].any()
    x[8] = 0
    # -0.0 and 0.0 are equal logits: the lower index first
    check(out, x, logits + 0.0, w1, w2, k, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_all_rows_masked_and_weights_of_idle_experts(dev, fmt):
    x, logits, w1, w2 = make(4, 6, 128, 128, fmt, 4, dev)
    logits[:, 3:] = -float("inf")
    want = gm.moe_layer_fwd(x, logits, w1, w2, 2)
    # NaN weights of experts nobody picks change nothing
    if fmt == "bf16":
        w1[3:], w2[3:] = float("nan"), float("nan")
    else:
        w1.scales[3:], w2.scales[3:] = 255, 255
    assert torch.equal(gm.moe_layer_fwd(x, logits, w1, w2, 2), want)
    logits[:] = -float("inf")
    out = gm.moe_layer_fwd(x, logits, w1, w2, 2)
    torch.cuda.synchronize()
    assert not out.any()


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_and_infinity_stay_in_their_token(dev, fmt):
    x, logits, w1, w2 = make(20, 4, 256, 128, fmt, 6, dev)
    want = gm.moe_layer_fwd(x, logits, w1, w2, 2)
    x[3, 7], x[11, 200] = float("nan"), float("inf")
    logits[15, 1] = float("inf")
    out = gm.moe_layer_fwd(x, logits, w1, w2, 2)
    torch.cuda.synchronize()
    bad = torch.zeros(20, dtype=torch.bool, device=dev)
    bad[[3, 11, 15]] = True
    assert torch.isnan(out[[3, 15]]).all() and not torch.isfinite(out[11]).any()
    assert torch.equal(out[~bad], want[~bad])


def test_agrees_with_the_grouped_path(dev):
    """MXFP8 weights: the same function as router, plan, GroupedMLP forward and
    combine, up to that path's bf16 rounding of each expert's rows."""
    T, E, k, H, F = 48, 8, 2, 512, 640
    g = torch.Generator(device=dev).manual_seed(8)
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    logits = torch.randn((T, E), generator=g, device=dev)
    w1 = (torch.randn((E, 2 * F, H), generator=g, device=dev) * H ** -0.5).bfloat16()
    w2 = (torch.randn((E, H, F), generator=g, device=dev) * F ** -0.5).bfloat16()
    out = gm.moe_layer_fwd(x, logits, quant(w1, "mxfp8"), quant(w2, "mxfp8"), k)
    ids, w = gm.router(logits, k)
    off, row_of, tok_of, r = gm.route_plan(ids, E, w)
    y, _ = gm.grouped_mlp_fwd(x[tok_of.long()].contiguous(), off, w1, w2, r)
    want = gm.combine(y, row_of)
    torch.cuda.synchronize()
    rel, row = O.parity_metrics(to64(out), to64(want))
    assert rel <= 1e-2 and row <= 5e-2, (rel, row)


@pytest.mark.parametrize("fmt", FMTS)
def test_graph_replays_follow_their_inputs(dev, fmt):
    T, E, k = 6, 8, 2
    x, logits, w1, w2 = make(T, E, 256, 384, fmt, 10, dev)
    gm.moe_layer_fwd(x, logits, w1, w2, k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gm.moe_layer_fwd(x, logits, w1, w2, k)
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn((T, 256), generator=g).bfloat16())
        logits.copy_(torch.randn((T, E), generator=g))
        logits[seed] = -float("inf")
        graph.replay()
        want = gm.moe_layer_fwd(x, logits, w1, w2, k)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_streams_at_once(dev):
    a = make(8, 16, 512, 512, "mxfp4", 20, dev)
    b = make(40, 16, 512, 512, "mxfp4", 21, dev)
    wa, wb = gm.moe_layer_fwd(*a, 4), gm.moe_layer_fwd(*b, 4)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s):
            outs.append((gm.moe_layer_fwd(*a, 4), wa))
        with torch.cuda.stream(t):
            outs.append((gm.moe_layer_fwd(*b, 4), wb))
    s.synchronize()
    t.synchronize()
    for got, want in outs:
        assert torch.equal(got, want)


def test_caller_owned_workspace_and_refusals(dev):
    x, logits, w1, w2 = make(4, 8, 256, 128, "mxfp4", 30, dev)
    want = gm.moe_layer_fwd(x, logits, w1, w2, 2)
    n = gm.lib().moe_layer_ws_bytes(gm.MX_DTYPE_MXFP4, 4, 8, 2, 256, 128)
    ws = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=dev)
    assert torch.equal(gm.moe_layer_fwd(x, logits, w1, w2, 2, ws=ws), want)
    assert (ws[n:] == 0xFF).all()
    with pytest.raises(gm.MxError, match="256-byte"):
        gm.moe_layer_fwd(x, logits, w1, w2, 2, ws=ws[16:])
    with pytest.raises(gm.MxError, match="status 2"):
        gm.moe_layer_fwd(x, logits, w1, w2, 9)
    with pytest.raises(TypeError, match="one format"):
        gm.moe_layer_fwd(x, logits, w1, gm.mxfp4_dequantize(w2), 2)
    with pytest.raises(ValueError, match="shape mismatch"):
        gm.moe_layer_fwd(x, logits[:, :7].contiguous(), w1, w2, 2)
    big = torch.zeros((129, 256), dtype=torch.bfloat16, device=dev)
    with pytest.raises(gm.MxError, match="exceeds 128 tokens"):
        gm.moe_layer_fwd(big, torch.zeros((129, 8), device=dev), w1, w2, 2)
    assert gm.moe_layer_fwd(x[:0], logits[:0], w1, w2, 2).shape == (0, 256)


def test_weights_past_4_gib(dev):
    """The last expert's rows of a weight of more than 2^32 bytes."""
    T, E, H, F = 2, 150, 2048, 8192
    w1 = torch.zeros((E, 2 * F, H), dtype=torch.uint8, device=dev)
    w2 = torch.zeros((E, H, F), dtype=torch.uint8, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: (torch.randn(s, generator=g, device=dev) * s[-1] ** -0.5).bfloat16()  # noqa: E731
    a, b = quant(rand(1, 2 * F, H), "mxfp8"), quant(rand(1, H, F), "mxfp8")
    w1[-1:], w2[-1:] = a.codes, b.codes
    s1 = torch.zeros((E, 2 * F, H // 32), dtype=torch.uint8, device=dev)
    s2 = torch.zeros((E, H, F // 32), dtype=torch.uint8, device=dev)
    s1[-1:], s2[-1:] = a.scales, b.scales
    x = torch.randn((T, H), generator=g, device=dev).bfloat16()
    logits = torch.full((T, E), -float("inf"), device=dev)
    logits[:, -1] = 0.5
    out = gm.moe_layer_fwd(x, logits, gm.MxTensor(w1, s1), gm.MxTensor(w2, s2), 2)
    want = gm.moe_layer_fwd(x, torch.zeros((T, 1), device=dev), a, b, 1)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and out.any()


def test_mxfp4_operators_together(dev):
    """A serving program's two ways through an MXFP4 layer, from one quantization
    of the weights: the grouped products over a prompt's rows, stage by stage,
    and the layer call for a step's tokens.

    Tolerance of the last comparison.  The grouped way rounds h to bf16 (twice
    2^-8 / (2 sqrt 3) in RMS: 1.6e-3 of a and of b) and z to bf16 (1.1e-3) before
    it quantizes z: z moves by about d = 2.5e-3 of itself.  A value that moves
    by d crosses an E4M3 step of s = 2^-4 .. 2^-3 of itself with probability d / s
    and then moves by s: sqrt(d s) = 1.3e-2 to 1.8e-2 in RMS.  y's own rounding
    adds 1e-3.  Twice the middle of that: 3e-2."""
    T, E, k, H, F = 96, 8, 2, 512, 640
    x, logits, w1, w2 = make(T, E, H, F, "bf16", 40, dev)
    q1, q2 = gm.mxfp4_quantize(w1)["row"], gm.mxfp4_quantize(w2)["row"]
    ids, w = gm.router(logits, k)
    off, row_of, tok_of, r = gm.route_plan(ids, E, w)
    xq = gm.permute_quantize(x, tok_of, off, T * k, colwise=False)["row"]
    h = gm.grouped_linear_fwd(xq, off, q1)
    a, b = h[:, :F].float(), h[:, F:].float()
    z = gm.mxfp8_quantize((r[:, None] * torch.nn.functional.silu(a) * b).bfloat16())["row"]
    y = gm.grouped_linear_fwd(z, off, q2)
    got = gm.combine(y, row_of)
    torch.cuda.synchronize()
    # the products, against their operands' values (2^-8 and the E4M3 term 2^-10 S)
    offs = off.cpu().numpy()
    for p, u, v in ((h, values(xq), values(q1)), (y, values(z), values(q2))):
        ref, S = O.grouped_linear(u, v, offs), O.grouped_linear(np.abs(u), np.abs(v), offs)
        assert (np.abs(to64(p) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * 2.0 ** -10 * S).all()
    # the weights the layer reads are the ones that dequantize to these values
    assert np.array_equal(to64(gm.mxfp4_dequantize(q1)), values(q1))
    out = gm.moe_layer_fwd(x, logits, q1, q2, k)
    torch.cuda.synchronize()
    check(out, x, logits, q1, q2, k, "mxfp4")
    rel, _ = O.parity_metrics(to64(got), to64(out))
    assert rel <= 3e-2, rel
