"""The bf16 GroupedLinear gradients and the adapter linear on the GPU at the limits of what
they take: the longest sums and rows, many experts in large tiles, scratch past 32 bits.

Operands are small whole numbers, so that every product and every sum, in any order, is a whole
number below 2^24 and exact in fp32 (and s A x, below 2^16, in its two bf16 parts): a result
is the exact one rounded once, and compared for equality."""

import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from tests.test_bf16_plans_host import DATA_GRAD, LARGE, WEIGHT_GRAD, plan  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def ints(g, *shape):
    """-2 .. 2, bf16."""
    return torch.randint(-2, 3, shape, generator=g, device=g.device, dtype=torch.int8).bfloat16()


def exact(a, b):
    """a @ b of whole numbers, in 64 bits (as slices of the sum where that is long)."""
    out = torch.zeros((a.shape[0], b.shape[1]), dtype=torch.float64, device=a.device)
    for k in range(0, a.shape[1], 1 << 16):
        out += a[:, k:k + (1 << 16)].double() @ b[k:k + (1 << 16)].double()
    return out


def check_grads(dy, x, w, off, dx, dw, r=None, dr=None, experts=None):
    for e in range(w.shape[0]) if experts is None else experts:
        rows = slice(off[e], off[e + 1])
        if dx is not None and off[e + 1] > off[e]:
            ref = exact(dy[rows], w[e])
            if r is not None:
                assert torch.equal(dr[rows].double(), (ref * x[rows].double()).sum(1))
                ref *= r[rows, None].double()
            assert torch.equal(dx[rows], ref.bfloat16())
        if dw is not None:
            d = dy[rows] if r is None else dy[rows] * r[rows, None].bfloat16()
            assert torch.equal(dw[e], exact(d.t(), x[rows]).to(dw.dtype))


@pytest.mark.parametrize("counts,N,K", [([1], 1 << 21, 32), ([1], 16, 1 << 21), ([100, 0, 200], 1 << 21, 32),
                                        ([100, 0, 200], 16, 1 << 21), ([5000000], 16, 32)])
def test_gradients_of_the_largest_sizes(dev, counts, N, K):
    g = torch.Generator(device=dev).manual_seed(N)
    off = torch.tensor([0] + counts).cumsum(0)
    M, E = int(off[-1]), len(counts)
    dy, x, w = ints(g, M, N), ints(g, M, K), ints(g, E, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        dx, dw, _ = gm.grouped_linear_bwd(dy, x, off.to(dev), w, dw_dtype=dtype)
        check_grads(dy, x, w, off.tolist(), dx, dw)
    old = torch.randint(-9, 9, w.shape, generator=g, device=dev).float()
    added = gm.grouped_linear_bwd(dy, x, off.to(dev), w, need_dx=False, dw=old.clone())[1]
    dw = gm.grouped_linear_bwd(dy, x, off.to(dev), w, need_dx=False, dw_dtype=torch.float32)[1]
    assert torch.equal(added, old + dw)


# experts up to the limit, in the large tiles of both products: full ones, empty ones, the last
# one full
@pytest.mark.parametrize("E,M,N,K", [(1000, 150000, 144, 4096), (1024, 262144, 272, 1056)])
def test_many_experts_in_large_tiles(dev, plan, E, M, N, K):  # noqa: F811
    assert plan(DATA_GRAD, E, M, M, K, N)[0] == LARGE and plan(WEIGHT_GRAD, E, M, N, K, M)[0] == LARGE
    g = torch.Generator(device=dev).manual_seed(E)
    share = torch.rand(E, generator=torch.Generator().manual_seed(E)) ** 3
    share[::7], share[-1] = 0, 1
    off = torch.cat([torch.zeros(1), (share.double().cumsum(0) / share.double().sum() * M).round()]).long()
    dy, x, w = ints(g, M, N), ints(g, M, K), ints(g, E, N, K)
    r = 2.0 ** torch.randint(-2, 2, (M,), generator=g, device=dev).float()
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, off.to(dev), w, row_scale=r, dw_dtype=torch.float32)
    check_grads(dy, x, w, off.tolist(), dx, dw, r, dr)


def test_an_added_gradient_past_32_bits(dev):
    """An fp32 gradient of 8.6 GB, added to: every expert's, the empty ones' kept."""
    E, N, K = 65, 4096, 8064
    g = torch.Generator(device=dev).manual_seed(0)
    off = [0, 40] + [40] * (E - 2) + [90]
    dy, x = ints(g, 90, N), ints(g, 90, K)
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev)     # (not read)
    dw = torch.full((E, N, K), 3.0, device=dev)
    gm.grouped_linear_bwd(dy, x, torch.tensor(off, device=dev), w, dw=dw, need_dx=False)
    for e in (0, E - 1):
        rows = slice(off[e], off[e + 1])
        assert torch.equal(dw[e], (exact(dy[rows].t(), x[rows]) + 3).float())
    assert (dw[1:E - 1] == 3).all()


@pytest.mark.parametrize("M,K,N,r,L", [
    (1, 1 << 21, 16, 16, 2), (16, 1 << 21, 32, 40, 5), (100, 1 << 21, 16, 16, 9), (1000, 1 << 20, 16, 16, 3),
    (1, 32, 1 << 21, 8, 2), (1, 2048, 1 << 21, 8, 2), (3, 4096, 1 << 20, 16, 3), (16, 32, 1 << 21, 8, 3),
    (100, 32, 1 << 21, 8, 3), (1000, 32, 1 << 20, 8, 3), (1000, 2112, 1 << 20, 8, 3)])
def test_adapter_linear_of_the_largest_sizes(dev, M, K, N, r, L):
    g = torch.Generator(device=dev).manual_seed(M + r)
    x, w = ints(g, M, K), ints(g, N, K)
    a, b = ints(g, L, r, K), ints(g, L, N, r).clamp_(-1, 1)
    ids = torch.randint(-1, L + 1, (M,), generator=g, device=dev).int()
    ids[0] = 0
    s = 2.0 ** torch.randint(-1, 2, (L,), generator=g, device=dev).float()
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    ref = exact(x, w.t())
    for l in range(L):
        rows = (ids == l).nonzero().flatten()
        h = exact(x[rows], a[l].t())
        assert h.numel() == 0 or h.abs().max() < 1 << 15
        ref[rows] += s[l].double() * (h @ b[l].double().t())
    assert ref.abs().max() < 1 << 23
    assert torch.equal(y, ref.float().bfloat16())


def test_low_rank_values_past_32_bits(dev):
    """17 million rows of rank 64: 4.4 GB of s A x."""
    g = torch.Generator(device=dev).manual_seed(4)
    M, K, N, r, L = 17000000, 32, 16, 64, 3
    x, w, a, b = ints(g, M, K), ints(g, N, K), ints(g, L, r, K), ints(g, L, N, r)
    ids = torch.randint(-1, L, (M,), generator=g, device=dev).int()
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    for at in (0, 8388608 - 500, 16777216 - 500, M - 1000):
        rows = slice(at, at + 1000)
        ref = exact(x[rows], w.t())
        for l in range(L):
            mine = ids[rows] == l
            ref[mine] += exact(x[rows][mine], a[l].t()) @ b[l].double().t()
        assert torch.equal(y[rows], ref.bfloat16())


@pytest.mark.parametrize("M", [1, 5, 16, 40, 300, 5001])
def test_ids_anywhere_outside(dev, M):
    g = torch.Generator(device=dev).manual_seed(M)
    K, N, r, L = 96, 272, 8, 4
    x, w, a, b = ints(g, M, K), ints(g, N, K), ints(g, L, r, K), ints(g, L, N, r)
    far = torch.tensor([-2 ** 31, -1, L, L + 1, 2 ** 31 - 1, 2 ** 30], dtype=torch.int32, device=dev)
    ids = far[torch.arange(M, device=dev) % 6].contiguous()
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    ref = exact(x, w.t())
    assert torch.equal(y, ref.bfloat16())
    ids[M // 2] = L - 1
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    ref[M // 2] += (exact(x[M // 2][None], a[-1].t()) @ b[-1].double().t())[0]
    assert torch.equal(y, ref.bfloat16())


@pytest.mark.parametrize("counts,N,K", [([300, 0, 200], 272, 416), ([4090], 2064, 4096), ([3, 0, 60], 4096, 14336)])
def test_gradients_on_two_streams_at_once(dev, counts, N, K):
    g = torch.Generator(device=dev).manual_seed(N)
    off = torch.tensor([0] + counts).cumsum(0).to(dev)
    M, E = sum(counts), len(counts)
    cases = [(ints(g, M, N), ints(g, M, K), off, ints(g, E, N, K)) for _ in range(2)]
    r = torch.rand(M, generator=g, device=dev)
    refs = [gm.grouped_linear_bwd(*c, row_scale=r) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], []
    for _ in range(4):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(gm.grouped_linear_bwd(*c, row_scale=r))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, refs[i % 2]))


def test_large_gradients_captured_and_replayed(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    counts, N, K = [5200, 0, 3000], 2064, 4128
    off = torch.tensor([0] + counts).cumsum(0).to(dev)
    M, E = sum(counts), len(counts)
    dy, x, w, r = ints(g, M, N), ints(g, M, K), ints(g, E, N, K), torch.rand(M, generator=g, device=dev)
    ws = torch.empty(gm.lib().grouped_linear_bwd_ws_bytes(E, M, N, K, 1), dtype=torch.uint8, device=dev)
    buf = torch.zeros(w.shape, device=dev)
    gm.grouped_linear_bwd(dy, x, off, w, row_scale=r, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, _, dr = gm.grouped_linear_bwd(dy, x, off, w, row_scale=r, dw=buf, ws=ws)
    for i in range(3):
        dy.copy_(ints(g, M, N))
        off.copy_(torch.tensor([0, 1000 * i, 5000, M], device=dev))
        buf.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = dx.clone(), buf.clone(), dr.clone()
        ref = gm.grouped_linear_bwd(dy, x, off, w, row_scale=r, dw_dtype=torch.float32)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
