"""The adapter linear on the GPU against FP64 (bounds: oracle/bf16_oracle.py)."""
import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import bf16_oracle as B

pytestmark = pytest.mark.gpu


def to64(t):
    return t.double().cpu().numpy()


def make(M, K, N, r, L, ids, seed, dev):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x = torch.where(torch.rand((M, K), generator=g) < 0.01, 20 * x, x).bfloat16()
    w = (torch.randn((N, K), generator=g) * 0.05).bfloat16()
    a = (torch.randn((L, r, K), generator=g) * K ** -0.5).bfloat16()
    b = (torch.randn((L, N, r), generator=g) * 0.3).bfloat16()
    s = torch.rand(L, generator=g) * 3 - 1
    if ids == "mixed":             # runs of one row, a few and many, some without an adapter
        out = []
        while len(out) < M:
            n = int(torch.randint(0, 6, (), generator=g)) ** 3 + 1
            out += [int(torch.randint(-1, L + 1, (), generator=g))] * n
        ids = out[:M]
    elif ids == "each":
        ids = torch.randint(-1, L, (M,), generator=g).tolist()
    elif isinstance(ids, int):
        ids = [ids] * M
    ids = torch.tensor(ids, dtype=torch.int32)
    return [t.to(dev) for t in (x, w, a, b, ids, s)]


def check(y, x, w, a, b, ids, s):
    x, w, a, b, ids = (to64(t) if t.is_floating_point() else t.cpu().numpy() for t in (x, w, a, b, ids))
    s = None if s is None else to64(s)
    err = np.abs(to64(y) - B.lora_fwd(x, w, a, b, ids, s))
    bound = B.lora_bound(x, w, a, b, ids, s)
    assert np.isfinite(err).all() and (err <= bound).all(), float((err - bound).max())


SHAPES = [
    (1, 32, 16, 8, 1, 0), (1, 4096, 256, 16, 3, 2), (1, 64, 48, 16, 2, -1), (2, 96, 16, 24, 2, "each"),
    (5, 1056, 80, 64, 9, "each"), (16, 512, 1040, 8, 20, "each"), (17, 160, 64, 128, 3, "each"),
    (33, 2048, 144, 40, 7, "mixed"), (64, 256, 128, 16, 64, "each"), (65, 288, 272, 32, 5, "mixed"),
    (100, 1024, 336, 8, 200, "each"), (130, 32, 2064, 16, 4, "mixed"), (257, 704, 528, 56, 6, "mixed"),
    (300, 544, 256, 512, 2, "mixed"), (515, 416, 1040, 16, 3, 1), (1000, 288, 784, 24, 8, "mixed"),
    (1500, 608, 1296, 32, 4, "mixed"), (700, 96, 2320, 8, 40, "each"),
    # sorted by adapter (eight rows an adapter on average), and the same unsorted
    (257, 96, 144, 8, 32, "each"), (600, 160, 528, 16, 75, "each"), (600, 160, 528, 16, 76, "each"),
    (1300, 1056, 272, 128, 3, "each"), (2049, 64, 2064, 24, 200, "each"),
    # enough tiles for the large kernel: whole rounds of 256 and what is left of them
    (4096, 64, 4096, 16, 3, "mixed"), (4200, 96, 4624, 24, 5, "mixed"), (5003, 288, 4112, 8, 70, "each"),
    (4400, 352, 4096, 64, 2, -1),
]


@pytest.mark.parametrize("M,K,N,r,L,ids", SHAPES)
def test_against_fp64(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, M + K + N, dev)
    nws = gm.lib().lora_linear_ws_bytes(M, N, K, L, r)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)     # NaN wherever it is read unwritten
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    y1 = gm.lora_linear_fwd(x, w, a, b, ids)
    torch.cuda.synchronize()
    check(y, x, w, a, b, ids, s)
    check(y1, x, w, a, b, ids, None)
    assert torch.equal(y, gm.lora_linear_fwd(x, w, a, b, ids, scale=s))     # one order of the sums


@pytest.mark.parametrize("M", [3, 40, 200, 1100])
def test_what_is_not_finite_stays_in_its_rows(dev, M):
    """An adapter that holds NaN and infinities, and a row of NaN: no other row changes."""
    x, w, a, b, ids, s = make(M, 288, 784, 16, 5, "mixed", M, dev)
    ids[0], ids[1], ids[2] = 0, 3, -1
    clean = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    b[3, 5, :], b[3, 700, 2], a[3, 1, 7] = float("nan"), float("inf"), float("-inf")
    x[2, 9] = float("nan")
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    torch.cuda.synchronize()
    hit = (ids == 3).cpu()
    hit[2] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert y[2].isnan().all() and y[1, 5].isnan()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 128, 129, 255, 256, 257])
def test_row_counts(dev, M):
    x, w, a, b, ids, s = make(M, 192, 320, 16, 4, "mixed", M, dev)
    y = torch.full((M + 8, 320), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(gm.lib().lora_linear_ws_bytes(M, 320, 192, 4, 16), dtype=torch.uint8, device=dev)
    st = gm.lib().lora_linear_fwd(x.data_ptr(), M, 192, w.data_ptr(), 320, a.data_ptr(), b.data_ptr(), 4, 16,
                                  ids.data_ptr(), s.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0, gm.last_error()
    torch.cuda.synchronize()
    check(y[:M], x, w, a, b, ids, s)
    assert (y[M:] == 7).all()                       # rows behind the last are left alone


@pytest.mark.parametrize("M", [1, 12, 100, 700])
def test_adapters_past_32_bits(dev, M):
    """b of 4.8 GB, a of 0.2: rows of the last adapters."""
    g = torch.Generator(device=dev).manual_seed(M)
    K, N, r, L = 512, 16400, 480, 305
    rnd = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.bfloat16)
    x, w, a = rnd(M, K), rnd(N, K), rnd(L, r, K)
    b = torch.empty((L, N, r), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    ids = (torch.arange(M, device=dev) % 3 + L - 3).int()
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    torch.cuda.synchronize()
    rows = torch.arange(0, M, max(1, M // 12), device=dev)
    check(y[rows], x[rows], w, a[-3:], b[-3:], ids[rows] - (L - 3), None)


def test_a_row_is_the_same_wherever_it_stands(dev):
    """Rows of a sorted batch in another order: the same bits for each row."""
    x, w, a, b, ids, s = make(900, 544, 784, 16, 6, "mixed", 5, dev)
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    for seed in range(3):
        p = torch.randperm(900, generator=torch.Generator().manual_seed(seed)).to(dev)
        assert torch.equal(gm.lora_linear_fwd(x[p], w, a, b, ids[p], scale=s), y[p])


@pytest.mark.parametrize("M", [4, 90, 900])
def test_captured_and_replayed(dev, M):
    x, w, a, b, ids, s = make(M, 544, 784, 16, 6, "mixed", M, dev)
    ws = torch.empty(gm.lib().lora_linear_ws_bytes(M, 784, 544, 6, 16), dtype=torch.uint8, device=dev)
    gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        ids.copy_(torch.randint(-1, 6, ids.shape, generator=g).int())
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        ref = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


# few rows of a wide layer: x in the LDS, columns by a CU in one stream (and the sizes next to
# those that take it)
WIDE = [
    (1, 2048, 12288, 16, 3, 2), (1, 2080, 12304, 32, 2, 0), (1, 2048, 12272, 16, 3, 1), (1, 2016, 12288, 16, 3, 1),
    (2, 2080, 16400, 16, 4, "each"), (2, 2112, 12304, 24, 4, "each"), (4, 2144, 12352, 8, 5, "each"),
    (5, 4096, 12304, 64, 9, "each"), (16, 4224, 12288, 8, 20, "each"), (16, 4256, 12288, 8, 20, "each"),
    (16, 2336, 14336, 64, 30, "each"), (3, 20000, 12288, 8, 2, "each"), (1, 2048, 28672, 512, 2, 1),
    (7, 2048, 12288, 16, 2, -1), (3, 4128, 12304, 24, 4, "each"), (16, 4128, 14336, 8, 20, "each"),
]


@pytest.mark.parametrize("M,K,N,r,L,ids", WIDE)
def test_wide_layers(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, M + K + N, dev)
    nws = gm.lib().lora_linear_ws_bytes(M, N, K, L, r)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=dev)
    st = gm.lib().lora_linear_fwd(x.data_ptr(), M, K, w.data_ptr(), N, a.data_ptr(), b.data_ptr(), L, r,
                                  ids.data_ptr(), s.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0, gm.last_error()
    torch.cuda.synchronize()
    check(y[:M], x, w, a, b, ids, s)
    assert (y[M] == 7).all()
    for _ in range(3):
        assert torch.equal(y[:M], gm.lora_linear_fwd(x, w, a, b, ids, scale=s))


@pytest.mark.parametrize("M,K,r", [(2, 2080, 16), (9, 4128, 40)])
def test_wide_layers_keep_what_is_not_finite(dev, M, K, r):
    x, w, a, b, ids, s = make(M, K, 12304, r, 3, "each", M, dev)
    ids[0], ids[1] = 1, -1
    clean = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    b[2] = float("nan")
    a[2] = float("inf")
    assert torch.equal(gm.lora_linear_fwd(x, w, a, b, ids, scale=s)[:2], clean[:2])
    x[1, K - 1] = float("nan")
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    torch.cuda.synchronize()
    assert torch.equal(y[0], clean[0]) and y[1].isnan().all()


# down projections in tiles: ranks over one column of tiles, adapters with few rows or none
@pytest.mark.parametrize("M,K,N,r,L,ids", [
    (2100, 96, 80, 136, 9, "mixed"), (1030, 1056, 48, 512, 3, "each"), (9000, 64, 32, 16, 700, "each"),
    (3000, 160, 144, 48, 5, "mixed"), (20000, 32, 16, 8, 40, "mixed"), (2060, 4128, 16, 64, 2, 1),
    (257, 544, 80, 512, 32, "each"), (4100, 64, 528, 40, 512, 511)])
def test_down_projection_in_tiles(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, M + K + N, dev)
    nws = gm.lib().lora_linear_ws_bytes(M, N, K, L, r)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    y1 = gm.lora_linear_fwd(x, w, a, b, ids)
    torch.cuda.synchronize()
    check(y, x, w, a, b, ids, s)
    check(y1, x, w, a, b, ids, None)
    p = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(dev)
    assert torch.equal(gm.lora_linear_fwd(x[p], w, a, b, ids[p], scale=s), y[p])


def test_down_projection_in_tiles_keeps_what_is_not_finite(dev):
    x, w, a, b, ids, s = make(1500, 288, 784, 96, 5, "mixed", 3, dev)
    ids[0], ids[1], ids[2] = 0, 3, -1
    clean = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    a[3, 1, 7], a[3, 90], b[3, 5, :] = float("-inf"), float("nan"), float("nan")
    x[2, 9] = float("nan")
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    torch.cuda.synchronize()
    hit = (ids == 3).cpu()
    hit[2] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert y[2].isnan().all() and y[1, 5].isnan()


# high ranks of few rows: sorted from 65 rows on, added in the join or in the tiles
@pytest.mark.parametrize("M,K,N,r,L,ids", [
    (72, 1056, 4096, 128, 16, "each"), (72, 1056, 4096, 128, 4, "each"), (64, 544, 2064, 256, 20, "mixed"),
    (65, 96, 1040, 512, 8, "each"), (200, 288, 4112, 64, 25, "each"), (255, 288, 4112, 40, 32, "each"),
    (256, 160, 4112, 40, 128, "each"), (257, 160, 4112, 40, 129, "each"), (20, 2080, 14336, 128, 30, "each")])
def test_high_ranks(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, M + K + N, dev)
    nws = gm.lib().lora_linear_ws_bytes(M, N, K, L, r)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    torch.cuda.synchronize()
    check(y, x, w, a, b, ids, s)
    assert torch.equal(y, gm.lora_linear_fwd(x, w, a, b, ids, scale=s))


# a long K in shares of middle tiles, more than a CU each: rows sorted, and as they are with
# the down projection beside the tiles
@pytest.mark.parametrize("L", [3, 90])
def test_shares_of_a_long_sum(dev, L):
    x, w, a, b, ids, s = make(700, 14336, 4096, 8, L, "each", L, dev)
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    torch.cuda.synchronize()
    check(y, x, w, a, b, ids, s)
    assert torch.equal(y, gm.lora_linear_fwd(x, w, a, b, ids, scale=s))


def test_two_streams_at_once(dev):
    cases = [make(M, 1024, 784, 16, 6, "mixed", M, dev) for M in (7, 300, 1500)]
    refs = [gm.lora_linear_fwd(x, w, a, b, ids, scale=s) for x, w, a, b, ids, s in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for st, (x, w, a, b, ids, s) in zip(streams, cases):
        with torch.cuda.stream(st):
            got.append([gm.lora_linear_fwd(x, w, a, b, ids, scale=s) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for ys, ref in zip(got, refs) for y in ys)


def test_adapters_trained_then_served(dev):
    """The operators together: adapters as two GroupedLinears over rows sorted by
    adapter, one step on their gradients, then served beside the shared projection in
    the batch's own order; the served rows against the trained weights in FP64."""
    g = torch.Generator().manual_seed(8)
    M, K, N, r, L = 240, 256, 288, 32, 4
    x, w, a, b, _, _ = make(M, K, N, r, L, 0, 8, dev)
    ids = torch.randint(-1, L, (M,), generator=g).int().to(dev)
    off, row_of, tok_of, _ = gm.route_plan(ids.view(M, 1), L)
    n = int(off[-1])
    xs = x[tok_of[:n].long()].contiguous()
    target = torch.randn((n, N), generator=g).bfloat16().to(dev)
    h = gm.grouped_linear_fwd(xs, off, a)
    dz = (gm.grouped_linear_fwd(h, off, b).float() - target.float()).bfloat16()
    dh, db, _ = gm.grouped_linear_bwd(dz, h, off, b, dw_dtype=torch.float32)
    _, da, _ = gm.grouped_linear_bwd(dh, xs, off, a, dw_dtype=torch.float32, need_dx=False)
    refb = B.linear_bwd(to64(dz), to64(h), to64(b), off.cpu().numpy())
    refa = B.linear_bwd(to64(dh), to64(xs), to64(a), off.cpu().numpy())
    for got, ref in ((db, refb[1]), (da, refa[1])):
        assert np.linalg.norm(to64(got) - ref) <= 1e-5 * np.linalg.norm(ref)
    a, b = (a.float() - 1e-3 * da).bfloat16(), (b.float() - 1e-3 * db).bfloat16()
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    torch.cuda.synchronize()
    check(y, x, w, a, b, ids, None)
