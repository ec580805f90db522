"""Gradients of the bf16 GroupedLinear on the GPU against FP64.

Bounds, element by element.  Products of two bf16 values are exact in fp32; a sum of
n of them in fp32, in any order and with truncation instead of rounding in places, is
off by at most n 2^-23 S, S the sum of their magnitudes.  A bf16 result adds half a
step (2^-8), a row scale one fp32 rounding (2^-24).  With row scales the weight
gradient's products take bf16(r dy) or bf16(r x): 2^-8 of each product's magnitude
more.  dr is a sum of K terms whose one factor is such a sum of N."""
import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import bf16_oracle as B

pytestmark = pytest.mark.gpu
N23 = 2.0 ** -23


def to64(t):
    return t.double().cpu().numpy()


def make(counts, N, K, seed, dev, scaled):
    g = torch.Generator().manual_seed(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    M, E = int(off[-1]), len(counts)
    dy = torch.randn((M, N), generator=g).bfloat16()
    x = torch.randn((M, K), generator=g)
    x = torch.where(torch.rand((M, K), generator=g) < 0.01, 20 * x, x).bfloat16()
    w = (torch.randn((E, N, K), generator=g) * 0.05).bfloat16()
    r = torch.rand(M, generator=g) - 0.25 if scaled else None
    return (dy.to(dev), x.to(dev), w.to(dev), off, torch.from_numpy(off).to(dev),
            None if r is None else r.to(dev))


def within(got, ref, bound):
    err = np.abs(to64(got) - ref)
    assert np.isfinite(err).all() and (err <= bound).all(), float((err - bound).max())


def check(dy, x, w, off, r, dx, dw, dr, old=None):
    a = [to64(t) for t in (dy, x, w)]
    rr = None if r is None else to64(r)
    ref = B.linear_bwd(*a, off, rr)
    mag = B.linear_bwd(*(np.abs(t) for t in a), off, None if rr is None else np.abs(rr))
    M, N, K = dy.shape[0], dy.shape[1], x.shape[1]
    if dx is not None:
        within(dx, ref[0], 2.0 ** -8 * np.abs(ref[0]) + (1 + 2.0 ** -8) * (N + 2) * N23 * mag[0])
    if dw is not None:
        most = int(np.diff(off).max()) if M else 0
        bound = (most + 2) * N23 * mag[1]
        if rr is not None:
            bound = (1 + 2.0 ** -7) * bound + (2.0 ** -8 + 2.0 ** -20) * mag[1]
        total = ref[1] if old is None else ref[1] + old
        if dw.dtype == torch.bfloat16:
            bound = 2.0 ** -8 * np.abs(total) + (1 + 2.0 ** -8) * bound
        elif old is not None:
            bound = bound + 2.0 ** -23 * (np.abs(total) + bound)
        within(dw, total, bound)
    if dr is not None:
        within(dr, ref[2], (N + K + 4) * N23 * mag[2])


SHAPES = [
    ([1], 16, 32),                              # the smallest
    ([1], 4096, 256),                           # one row, a long sum for dx
    ([3, 0, 1, 0, 0, 2], 48, 96),               # empty experts, sums that end inside a step
    ([64], 64, 128),                            # whole small tiles
    ([65, 63, 1], 80, 160),                     # one over, one under
    ([16], 1040, 32),
    ([130, 0, 7], 272, 416),
    ([300, 0, 17, 511], 336, 256),
    ([0, 0, 9, 0], 1408, 704),
    ([700], 32, 1024),                          # an adapter's own gradient
    ([2000, 5], 16, 2048),                      # long sums for dw, few tiles
    ([256, 1, 255, 257], 512, 544),
    ([1200, 333, 800], 1040, 1312),
    ([2, 1500, 40, 0, 0, 700], 2064, 288),
]


# enough tiles for the large kernel: whole rounds of 256 and what is left of them, sums
# of one, two and three steps, ragged edges on every side
LARGE = [
    ([4097], 16, 4128), ([2500, 0, 3, 1700, 300], 80, 4096), ([4000, 130, 257], 208, 4384),
    ([900, 0, 5000, 129], 144, 4640), ([0, 70, 129, 700, 0, 1], 2064, 2848), ([1500, 10], 4112, 3616),
]
# weight gradients of the large kernel: one expert's round, and many experts' chains of
# sums of no, one, two and more steps
LARGE_W = [([700], 3600, 3616), (([0, 1, 64, 65, 0, 0, 129, 200, 3, 300] * 4)[:32], 16, 8192),
           (([70, 0, 1, 128, 0, 333, 40] * 5)[:31], 272, 4128)]


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("counts,N,K", SHAPES + LARGE + LARGE_W)
def test_against_fp64(dev, counts, N, K, scaled):
    dy, x, w, off, offd, r = make(counts, N, K, N + K, dev, scaled)
    nws = gm.lib().grouped_linear_bwd_ws_bytes(len(counts), x.shape[0], N, K, scaled)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, ws=ws)
    dx2, dw2, dr2 = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, dw_dtype=torch.float32)
    dx3, none, dr3 = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, need_dw=False)
    torch.cuda.synchronize()
    check(dy, x, w, off, r, dx, dw, dr)
    check(dy, x, w, off, r, None, dw2, None)
    # one order of the sums, whatever is asked for beside
    assert torch.equal(dx, dx2) and torch.equal(dx, dx3) and torch.equal(dw2.bfloat16(), dw) and none is None
    assert (dr is None and dr2 is None) if r is None else torch.equal(dr, dr2) and torch.equal(dr, dr3)
    for e, c in enumerate(counts):
        assert c or not dw[e].any()


@pytest.mark.parametrize("scaled", [False, True])
def test_shares_of_a_long_sum(dev, scaled):
    """dx over a long N, cut into shares of middle tiles."""
    dy, x, w, off, offd, r = make([690, 10], 14336, 2048, 7, dev, scaled)
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    dx1, _, dr1 = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, need_dw=False)
    torch.cuda.synchronize()
    check(dy, x, w, off, r, dx, dw, dr)
    assert torch.equal(dx, dx1) and (r is None or torch.equal(dr, dr1))


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 1], 48, 96), ([300, 0, 17, 511], 336, 256),
                                        ([2000, 5], 16, 2048)] + LARGE_W)
def test_adding_to_a_gradient_buffer(dev, counts, N, K, scaled):
    dy, x, w, off, offd, r = make(counts, N, K, 3 * N + K, dev, scaled)
    buf = torch.randn(w.shape, generator=torch.Generator().manual_seed(1)).to(dev)
    old = buf.clone()
    _, dw, _ = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, dw=buf, need_dx=False)
    torch.cuda.synchronize()
    assert dw is buf
    check(dy, x, w, off, r, None, dw, None, to64(old))
    for e, c in enumerate(counts):
        assert c or torch.equal(buf[e], old[e])


def test_no_rows(dev):
    w = torch.ones((3, 16, 32), dtype=torch.bfloat16, device=dev)
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    dy, x = (torch.empty((0, c), dtype=torch.bfloat16, device=dev) for c in (16, 32))
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, off, w, row_scale=torch.empty(0, device=dev))
    assert dx.shape == (0, 32) and not dw.any() and dr.shape == (0,)
    buf = torch.ones((3, 16, 32), device=dev)
    gm.grouped_linear_bwd(dy, x, off, w, dw=buf)
    assert (buf == 1).all()
    assert gm.grouped_linear_bwd(dy, x, off, w, need_dw=False)[1] is None


def test_many_experts(dev):
    g = torch.Generator().manual_seed(2)
    counts = torch.randint(0, 3, (1024,), generator=g).tolist()
    dy, x, w, off, offd, r = make(counts, 32, 64, 9, dev, True)
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    torch.cuda.synchronize()
    check(dy, x, w, off, r, dx, dw, dr)


@pytest.mark.parametrize("counts,N,K", [([40, 0, 30], 80, 96), ([700, 0, 600], 528, 544)])
def test_only_what_is_asked_for_is_written(dev, counts, N, K):
    """Outputs at the front of longer buffers, through the C entry: what lies behind
    them, and outputs that are not asked for, stay as they were."""
    dy, x, w, off, offd, r = make(counts, N, K, 4, dev, True)
    M, E, L = x.shape[0], len(counts), gm.lib()
    nws = L.grouped_linear_bwd_ws_bytes(E, M, N, K, 1)
    ws = torch.full((nws + 256,), 7, dtype=torch.uint8, device=dev)
    mark = 1234.0
    bufs = {"dx": torch.full((M * K + 4096,), mark, dtype=torch.bfloat16, device=dev),
            "dr": torch.full((M + 1024,), mark, device=dev),
            "dw": torch.full((w.numel() + 4096,), mark, dtype=torch.bfloat16, device=dev)}
    sizes = {"dx": M * K, "dr": M, "dw": w.numel()}
    keep = {n: bufs[n][0].item() for n in bufs}

    def call(*names):
        for b in bufs.values():
            b.fill_(mark)
        at = {n: bufs[n].data_ptr() if n in names else 0 for n in bufs}
        st = L.grouped_linear_bwd(dy.data_ptr(), x.data_ptr(), offd.data_ptr(), E, M, w.data_ptr(), N, K,
                                  r.data_ptr(), at["dx"], at["dr"], at["dw"], 0, ws.data_ptr(), nws,
                                  torch.cuda.current_stream().cuda_stream)
        assert st == 0, gm.last_error()
        torch.cuda.synchronize()
        for n, b in bufs.items():
            assert (b[sizes[n] if n in names else 0:] == keep[n]).all(), (names, n)
        assert (ws[nws:] == 7).all()

    for names in (("dx", "dr", "dw"), ("dx",), ("dx", "dr"), ("dw",)):
        call(*names)
        check(dy, x, w, off, r, bufs["dx"][:M * K].view(M, K) if "dx" in names else None,
              bufs["dw"][:w.numel()].view(E, N, K) if "dw" in names else None,
              bufs["dr"][:M] if "dr" in names else None)


@pytest.mark.parametrize("counts,N,K", [([5, 70, 3], 80, 96), ([600, 3, 500], 528, 544)])
def test_what_is_not_finite_stays_in_its_row_and_expert(dev, counts, N, K):
    dy, x, w, off, offd, r = make(counts, N, K, 6, dev, True)
    clean = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    dy[1, 3], x[1, 7], w[2, N - 1, K - 1] = float("nan"), float("inf"), float("-inf")
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    torch.cuda.synchronize()
    fine = torch.ones(x.shape[0], dtype=torch.bool)
    fine[1] = False
    fine[off[2]:] = False
    assert torch.equal(dx[fine], clean[0][fine]) and torch.equal(dr[fine], clean[2][fine])
    assert dx[1].isnan().all() and torch.equal(dx[off[2]:, :K - 1], clean[0][off[2]:, :K - 1])
    assert torch.equal(dw[1:], clean[1][1:])
    assert dw[0, 3].isnan().all() and not dw[0, :, 7].isfinite().any()
    keep = torch.ones(N, dtype=torch.bool)
    keep[3] = False
    assert torch.equal(dw[0][keep][:, :7], clean[1][0][keep][:, :7])


def test_offsets_past_32_bits(dev):
    """x and dx of 4.4 GB, then weights and their gradient of 4.3 GB: the last rows and the
    last expert."""
    g = torch.Generator(device=dev).manual_seed(3)
    M, N, K = 270000, 16, 8192
    x = torch.randn((M, K), generator=g, device=dev, dtype=torch.bfloat16)
    dy = torch.randn((M, N), generator=g, device=dev, dtype=torch.bfloat16)
    w = torch.randn((2, N, K), generator=g, device=dev, dtype=torch.bfloat16)
    off = np.array([0, M - 300, M])
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, torch.from_numpy(off).to(dev), w,
                                       row_scale=torch.ones(M, device=dev))
    tail = slice(M - 300, M)
    check(dy[tail], x[tail], w[1:], np.array([0, 300]), torch.ones(300), dx[tail], dw[1:], dr[tail])
    del x, dx, dy, dw, dr
    E, N, K = 65, 4096, 8064
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    off = np.array([0] * (E - 1) + [3, 50])
    x = torch.randn((50, K), generator=g, device=dev, dtype=torch.bfloat16)
    dy = torch.randn((50, N), generator=g, device=dev, dtype=torch.bfloat16)
    dx, dw, _ = gm.grouped_linear_bwd(dy, x, torch.from_numpy(off).to(dev), w)
    check(dy[3:], x[3:], w[-1:], np.array([0, 47]), None, dx[3:], dw[-1:], None)
    assert not dw[0].any() and not dw[E - 3].any()


@pytest.mark.parametrize("counts,N,K", [([33, 0, 60], 80, 96), ([900, 300], 784, 544)])
def test_captured_and_replayed(dev, counts, N, K):
    dy, x, w, off, offd, r = make(counts, N, K, 11, dev, True)
    ws = torch.empty(gm.lib().grouped_linear_bwd_ws_bytes(len(counts), x.shape[0], N, K, 1), dtype=torch.uint8,
                     device=dev)
    buf = torch.zeros(w.shape, device=dev)
    gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, _, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, dw=buf, ws=ws)
    for i in range(3):
        dy.copy_(torch.randn(dy.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        buf.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = dx.clone(), buf.clone(), dr.clone()
        ref = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, dw_dtype=torch.float32)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_on_another_stream(dev):
    dy, x, w, off, offd, r = make([500, 100], 256, 512, 12, dev, True)
    ref = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
