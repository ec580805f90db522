"""GroupedLinear on MXFP4 weights (x MXFP4 or MXFP8) on the GPU against the
FP64 product of the very values that the codes stand for.

Bound, element by element.  The products of two E2M1 or E4M3 values with
power-of-two scales are exact in fp32; a sum of K of them in fp32, in any
order and with truncation instead of rounding in places, is off by at most
K 2^-23 S, S the sum of the products' magnitudes; a row scale adds one
rounding (2^-24) and the bf16 result half a step (2^-8), both relative.

With an E4M3 operand the matrix instruction itself is coarser: it aligns the
eight products of each run of eight K values to the largest of them and drops
what lies below 2^-13 of that (test_products_of_a_run_of_eight_are_aligned
measures it; E2M1 products span less than 2^8 and lose nothing).  Each product
of a run then loses less than 2^-13 of the run's largest, p: a run loses less
than 8 * 2^-13 p = 2^-10 p, and since the runs' largest products sum to at most
S, the whole sum less than 2^-10 S."""
import re

import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import mx4_oracle as P
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


def values(q):
    c, s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    return P.dequantize4_lastdim(c, s) if isinstance(q, gm.Mx4Tensor) else O.dequantize_lastdim(c, s)


def assert_close(y, x, w, off, r=None, fmt="mxfp4"):
    """y bf16 against x [M, K] . w [E, N, K]^T of float64 values, x held as fmt."""
    ref = O.grouped_linear(x, w, off)
    S = O.grouped_linear(np.abs(x), np.abs(w), off)
    if r is not None:
        rr = r.cpu().numpy().astype(np.float64)[:, None]
        ref, S = ref * rr, S * np.abs(rr)
    K = x.shape[1]
    part = (K + 2) * 2.0 ** -23 + (2.0 ** -10 if fmt == "mxfp8" else 0.0)
    bound = 2.0 ** -8 * np.abs(ref) + part * (1 + 2.0 ** -8) * S
    err = np.abs(to64(y) - ref)
    assert (err <= bound).all(), float((err - bound).max())


def make(counts, K, N, seed, fmt, dev):
    g = torch.Generator().manual_seed(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M, E = int(off[-1]), len(counts)
    x = torch.randn((M, K), generator=g)
    x = torch.where(torch.rand((M, K), generator=g) < 0.01, 50 * x, x).bfloat16()
    w = (torch.randn((E, N, K), generator=g) * 0.05).bfloat16()
    xq = (gm.mxfp4_quantize if fmt == "mxfp4" else gm.mxfp8_quantize)(x.to(dev))["row"]
    wq = gm.mxfp4_quantize(w.to(dev))["row"]
    r = torch.rand(M, generator=g).to(dev)
    return xq, wq, off, torch.from_numpy(off).to(dev), r


SHAPES = [
    ([1], 128, 32),                             # one row
    ([1], 4096, 256),
    ([3, 0, 1, 0, 0, 2], 256, 96),              # empty experts, N tail
    ([16], 512, 64),                            # one full column tile
    ([17], 640, 64),                            # one row over
    ([33, 5, 64, 65, 130], 384, 160),           # every tile count, chunks of rows
    ([0, 0, 7, 0], 1408, 2816),
    ([300, 0, 17, 511], 256, 320),              # many rows an expert, ragged
    ([256, 1, 255, 257], 512, 544),
    ([700], 1024, 288),
    ([0, 2000, 3], 2048, 96),
    # K not a multiple of 128
    ([5], 32, 32), ([2, 0, 40], 96, 64), ([70, 1], 160, 96), ([16, 16], 544, 128),
    ([9, 200], 1056, 64), ([3], 4064, 32),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_against_the_product_of_the_codes(dev, counts, K, N, fmt):
    xq, wq, off, offd, r = make(counts, K, N, K + N + len(counts), fmt, dev)
    y = gm.grouped_linear_fwd(xq, offd, wq)
    ys = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    x, w = values(xq), values(wq)
    assert_close(y, x, w, off, fmt=fmt)
    assert_close(ys, x, w, off, r, fmt=fmt)
    assert torch.equal(y, gm.grouped_linear_fwd(xq, offd, wq))       # one order of the sums


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_every_code_and_many_scales(dev, fmt):
    """Codes drawn over all patterns (E4M3 without its NaN), scales over 2^-40 .. 2^40."""
    g = torch.Generator().manual_seed(9)
    M, E, N, K = 100, 3, 96, 512
    wq = gm.Mx4Tensor(torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8).to(dev),
                      torch.randint(87, 168, (E, N, K // 32), generator=g, dtype=torch.uint8).to(dev))
    xs = torch.randint(87, 168, (M, K // 32), generator=g, dtype=torch.uint8).to(dev)
    if fmt == "mxfp4":
        xq = gm.Mx4Tensor(torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8).to(dev), xs)
    else:
        c = torch.randint(0, 256, (M, K), generator=g, dtype=torch.uint8)
        c[(c & 127) == 127] = 0
        xq = gm.MxTensor(c.to(dev), xs)
    off = np.array([0, 40, 40, 100])
    y = gm.grouped_linear_fwd(xq, torch.from_numpy(off).to(dev), wq)
    torch.cuda.synchronize()
    assert_close(y, values(xq), values(wq), off, fmt=fmt)


def test_products_of_a_run_of_eight_are_aligned(dev):
    """The hardware fact behind the E4M3 bound: 256 * 4 - 256 * 4 + p in one run
    of eight keeps p down to 2^-13 of the large products; in different runs, p
    is kept much further down."""
    def dot(at, p):
        x = torch.zeros(1, 128)
        w = torch.zeros(1, 32, 128)
        x[0, 0], w[:, :, 0] = 256.0, 4.0
        x[0, 1], w[:, :, 1] = -256.0, 4.0
        x[0, at], w[:, :, at] = p, 1.0
        e4 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).to(dev)  # noqa: E731
        one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=dev)  # noqa: E731
        wq = gm.mxfp4_quantize(w.bfloat16().to(dev))["row"]
        y = gm.grouped_linear_fwd(gm.MxTensor(e4(x), one(1, 4)), torch.tensor([0, 1], device=dev), wq)
        return float(y[0, 0])
    big = 256.0 * 4.0
    for d in range(2, 14):          # p from 256 down; E4M3 ends at 448
        assert dot(2, big * 2.0 ** -d) == big * 2.0 ** -d, d
    for d in range(2, 20):
        assert dot(40, big * 2.0 ** -d) == big * 2.0 ** -d, d


def test_the_alignment_drops_what_lies_below(dev):
    """The other side of that fact: within the run of eight, a product is cut
    toward zero to a multiple of 2^-13 of the large ones; the next run is not
    touched."""
    e4 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).to(dev)  # noqa: E731
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=dev)  # noqa: E731
    w = torch.zeros(1, 32, 128)
    w[:, :, :2], w[:, :, 2:16] = 4.0, 1.0
    wq = gm.mxfp4_quantize(w.bfloat16().to(dev))["row"]
    grid = 256.0 * 4.0 * 2.0 ** -13
    # (place among the K values, value, what is left of it); E4M3 ends at 2^-9
    cases = [(at, sign * p, sign * (p // grid * grid if at < 8 else p))
             for at in (2, 7, 8, 15) for sign in (1.0, -1.0)
             for p in (1.75, 0.9375, 0.1875, 0.125, 0.1171875, 0.0625, 0.015625, 2.0 ** -9)]
    x = torch.zeros(len(cases), 128)
    x[:, 0], x[:, 1] = 256.0, -256.0
    for i, (at, p, _) in enumerate(cases):
        x[i, at] = p
    off = torch.tensor([0, len(cases)], device=dev)
    y = gm.grouped_linear_fwd(gm.MxTensor(e4(x), one(len(cases), 4)), off, wq)
    torch.cuda.synchronize()
    assert y[:, 0].tolist() == [left for _, _, left in cases]
    assert torch.equal(y, y[:, :1].expand_as(y))


@pytest.mark.parametrize("M", [5, 400])
def test_nan_blocks_stay_in_their_row_and_column(dev, M):
    xq, wq, off, offd, _ = make([M, 3], 512, 160, 4, "mxfp4", dev)
    clean = gm.grouped_linear_fwd(xq, offd, wq)
    xq.scales[2, 7] = 255                  # a NaN block of row 2
    wq.scales[0, 33, 0] = 255              # and one of expert 0's column 33
    y = gm.grouped_linear_fwd(xq, offd, wq)
    torch.cuda.synchronize()
    bad = torch.zeros(y.shape, dtype=torch.bool, device=dev)
    bad[2] = True
    bad[:M, 33] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts", [[3, 0, 6], [200, 0, 140]])
def test_data_gradient_from_the_columnwise_copy(dev, counts, fmt):
    """dX = dY . W[e] as the same call on the columnwise weight copy: against
    the formula, and against differences of the (linear) forward product."""
    g = torch.Generator().manual_seed(len(fmt) + counts[0])
    K, N, E = 256, 384, len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    offd = torch.from_numpy(off).to(dev)
    M = int(off[-1])
    # weights and gradients that both copies hold exactly: small whole values
    w = torch.randint(-3, 4, (E, N, K), generator=g).float()
    w[..., ::32, :] = 4.0
    w[..., ::32] = 4.0
    wq = gm.mxfp4_quantize(w.bfloat16().to(dev), rowwise=True, colwise=True)
    dy = torch.randint(-3, 4, (M, N), generator=g).float()
    dy[:, ::32] = 6.0
    q = gm.mxfp4_quantize if fmt == "mxfp4" else gm.mxfp8_quantize
    dyq = q(dy.bfloat16().to(dev))["row"]
    dx = gm.grouped_linear_fwd(dyq, offd, wq["col"])
    torch.cuda.synchronize()
    wt = np.swapaxes(w.numpy().astype(np.float64), 1, 2)
    assert np.array_equal(values(wq["col"]), wt)
    assert_close(dx, dy.numpy().astype(np.float64), wt, off, fmt=fmt)
    # <dY, f(x + h) - f(x)> = <dX, h> for one changed element at a time
    x = torch.zeros((M, K))
    x[:, ::32] = 4.0
    base = to64(gm.grouped_linear_fwd(q(x.bfloat16().to(dev))["row"], offd, wq["row"]))
    for row, col in ((0, 1), (M - 1, K - 1), (M // 2, 37)):
        x2 = x.clone()
        x2[row, col] += 2.0
        y2 = to64(gm.grouped_linear_fwd(q(x2.bfloat16().to(dev))["row"], offd, wq["row"]))
        diff = float((dy.numpy().astype(np.float64) * (y2 - base)).sum()) / 2.0
        # y2 - base = 2 w exactly up to the bf16 rounding of y's row: half a
        # step of each element, weighted with |dy|
        tol = float((np.abs(dy.numpy()[row]) * (np.abs(y2[row]) + np.abs(base[row]))).sum()) * 2.0 ** -8 / 2.0
        tol += abs(float(dx[row, col])) * 2.0 ** -8
        assert abs(diff - float(dx[row, col])) <= tol


def test_operand_past_4_gib(dev):
    """Weights of more than 2^32 bytes: the last expert's rows are read where they lie."""
    E, N, K = 40, 8192, 32768
    w = gm.Mx4Tensor(torch.zeros((E, N, K // 2), dtype=torch.uint8, device=dev),
                     torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=dev))
    g = torch.Generator(device=dev).manual_seed(0)
    w.codes[-1] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=dev)
    x = torch.randn((600, K), generator=g, device=dev).bfloat16()
    for M in (3, 600):
        off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
        off[-1] = M
        xq = gm.mxfp4_quantize(x[:M].contiguous())["row"]
        y = gm.grouped_linear_fwd(xq, off, w)
        last = gm.Mx4Tensor(w.codes[-1:, :64].contiguous(), w.scales[-1:, :64].contiguous())
        assert_close(y[:, :64], values(xq), values(last), np.array([0, M]))
        end = gm.Mx4Tensor(w.codes[-1:, -64:].contiguous(), w.scales[-1:, -64:].contiguous())
        assert_close(y[:, -64:], values(xq), values(end), np.array([0, M]))


@pytest.mark.parametrize("counts", [[2, 5, 0, 9], [300, 0, 150, 40]])
def test_graph_replays_follow_their_inputs(dev, counts):
    xq, wq, off, offd, r = make(counts, 512, 288, 11, "mxfp8", dev)
    y = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    M = int(off[-1])
    for seed in (1, 2, 3):
        g = torch.Generator().manual_seed(seed)
        cut = torch.sort(torch.randint(0, M + 1, (len(counts) - 1,), generator=g)).values
        offd[1:-1] = cut.to(dev)
        xq.codes.copy_(torch.randint(0, 120, xq.codes.shape, generator=g, dtype=torch.uint8))
        r.copy_(torch.rand(M, generator=g))
        graph.replay()
        want = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_another_stream(dev):
    xq, wq, off, offd, r = make([20, 300], 512, 96, 12, "mxfp4", dev)
    want = gm.grouped_linear_fwd(xq, offd, wq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = gm.grouped_linear_fwd(xq, offd, wq)
    s.synchronize()
    assert torch.equal(y, want)


def test_no_rows_and_bad_operands(dev):
    xq, wq, off, offd, r = make([4, 4], 128, 64, 13, "mxfp4", dev)
    none = gm.Mx4Tensor(xq.codes[:0], xq.scales[:0])
    assert gm.grouped_linear_fwd(none, torch.zeros(3, dtype=torch.int64, device=dev), wq).shape == (0, 64)
    with pytest.raises(TypeError):
        gm.grouped_linear_fwd(torch.zeros((8, 128), dtype=torch.bfloat16, device=dev), offd, wq)
    with pytest.raises(TypeError):
        gm.grouped_linear_fwd(xq, offd, torch.zeros((2, 64, 128), dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError, match="K mismatch"):
        gm.grouped_linear_fwd(gm.mxfp4_quantize(torch.zeros((8, 160), dtype=torch.bfloat16, device=dev))["row"],
                              offd, wq)
    with pytest.raises(ValueError, match="scales"):
        gm.grouped_linear_fwd(gm.Mx4Tensor(xq.codes, xq.scales[:, :2].contiguous()), offd, wq)
    with pytest.raises(ValueError, match="offsets"):
        gm.grouped_linear_fwd(xq, offd[:2].contiguous(), wq)
    with pytest.raises(ValueError, match="row_scale"):
        gm.grouped_linear_fwd(xq, offd, wq, row_scale=r[:3].contiguous())


def test_mx_check_refuses_bad_offsets(dev, monkeypatch):
    xq, wq, off, offd, _ = make([4, 4], 128, 64, 14, "mxfp8", dev)
    monkeypatch.setenv("MX_CHECK", "1")
    gm.grouped_linear_fwd(xq, offd, wq)
    for bad, msg in (([0, 9, 8], "decrease"), ([0, 4, 7], "row count"), ([1, 4, 8], "offsets[0]")):
        with pytest.raises(gm.MxError, match=re.escape(msg)):
            gm.grouped_linear_fwd(xq, torch.tensor(bad, dtype=torch.int64, device=dev), wq)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 1024])
def test_more_tiles_than_workgroups(dev, K, fmt):
    """324 and more tiles of 256 x 256 on 256 workgroups: each runs a chain
    whose last K steps load the next tile's first ones; one to eight K steps,
    whole and half ones, odd and even."""
    xq, wq, off, offd, r = make([9000, 37, 0, 11000, 5], K, 1024 - 32, K, fmt, dev)
    y = gm.grouped_linear_fwd(xq, offd, wq)
    ys = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    x, w = values(xq), values(wq)
    assert_close(y, x, w, off, fmt=fmt)
    assert_close(ys, x, w, off, r, fmt=fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts,K,N", [
    ([9000], 2080, 32),             # one expert, one column block, 141 turns
    ([700, 0, 1300, 1], 1056, 160),
    ([65, 4000, 3], 4064, 96),
    ([2048] + [0] * 63, 512, 8192),     # whole K: an average of 32 rows, all on one expert
    ([1, 0, 1985] + [1] * 30, 160, 544),
])
def test_many_turns_of_an_expert(dev, counts, K, N, fmt):
    """Experts whose rows take many turns of the weight stream."""
    xq, wq, off, offd, r = make(counts, K, N, K + N, fmt, dev)
    y = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    assert_close(y, values(xq), values(wq), off, r, fmt=fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("most,K,N", [
    (8, 512, 160),          # one tile of rows a turn, for experts with more
    (34, 256, 160),         # rows as a weight stream, up to several turns
    (140, 256, 160),        # tiles of 256 x 256, one column of them
    (34, 256, 2112),        # and nine
])
def test_many_uneven_experts(dev, most, K, N, fmt):
    """64 experts with most rows on average, from none to ten times that."""
    rng = np.random.default_rng(most + N)
    counts = rng.multinomial(most * 64, rng.dirichlet(np.full(64, 0.4)))
    xq, wq, off, offd, r = make(counts.tolist(), K, N, most, fmt, dev)
    y = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    assert_close(y, values(xq), values(wq), off, r, fmt=fmt)


def test_graph_replays_of_tiles(dev):
    """Captured 256 x 256 tiles follow their offsets, empty experts among them."""
    xq, wq, off, offd, r = make([400, 100, 300, 2], 512, 288, 21, "mxfp4", dev)
    want0 = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
    for cut in ([400, 500, 800], [0, 0, 0], [802, 802, 802], [1, 257, 513], [400, 500, 800]):
        offd[1:4] = torch.tensor(cut, device=dev)
        graph.replay()
        want = gm.grouped_linear_fwd(xq, offd, wq, row_scale=r)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert torch.equal(y, want0)


@pytest.mark.parametrize("fmt,M,N,K", [
    ("mxfp4", 3, 32, 1 << 26), ("mxfp8", 17, 32, 1 << 26), ("mxfp4", 3, 32, (1 << 26) - 32),
    ("mxfp4", 200, 64, (1 << 24) - 128), ("mxfp8", 200, 64, (1 << 23) - 128),
])
def test_longest_rows(dev, fmt, M, N, K):
    """The largest K of either kernel: weights of zeros but for both ends of their rows."""
    g = torch.Generator(device=dev).manual_seed(K % 97)
    ends = [slice(0, 256), slice(K - 256, K)]
    w = gm.Mx4Tensor(torch.zeros((1, N, K // 2), dtype=torch.uint8, device=dev),
                     torch.full((1, N, K // 32), 127, dtype=torch.uint8, device=dev))
    bits = 4 if fmt == "mxfp4" else 8
    x = (gm.Mx4Tensor if fmt == "mxfp4" else gm.MxTensor)(
        torch.full((M, K * bits // 8), 0x21, dtype=torch.uint8, device=dev),
        torch.full((M, K // 32), 127, dtype=torch.uint8, device=dev))
    small = lambda n: torch.randint(0, 112, n, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    xe, we = [], []
    for e in ends:
        at = slice(e.start // 2, e.stop // 2)
        xat = at if fmt == "mxfp4" else e
        w.codes[:, :, at] = small((1, N, 128))
        x.codes[:, xat] = small((M, xat.stop - xat.start))
        xe.append(values(type(x)(x.codes[:, xat].contiguous(), x.scales[:, :8].contiguous())))
        we.append(values(gm.Mx4Tensor(w.codes[:, :, at].contiguous(), w.scales[:, :, :8].contiguous())))
    off = np.array([0, M])
    y = gm.grouped_linear_fwd(x, torch.from_numpy(off).to(dev), w)
    torch.cuda.synchronize()
    assert_close(y, np.concatenate(xe, 1), np.concatenate(we, 2), off, fmt=fmt)
