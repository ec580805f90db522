"""The 256 x 256 tiles of the bf16 products on the GPU against FP64: the adapter linear and the
data gradient at sizes whose plan is the large kernel (test_bf16_plans_host.py asks the planner),
and the down projection of many unsorted rows.

References and bounds are those of oracle/bf16_oracle.py and test_gpu_linear_bwd.py, computed
in 64 bits by torch on the GPU, as the sizes need."""
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm

pytestmark = pytest.mark.gpu
N23, H = 2.0 ** -23, 2.0 ** -8


# (M, K, N, r, L, ids): runs "mixed" of one row, a few and many, "each" row for itself, "pairs"
# of one or two adapters for a hundred rows, or one id for all
FORWARD = [
    (4096, 1504, 4096, 16, 3, "mixed"),         # one whole round, K % 64 == 32
    (5001, 2080, 4112, 24, 5, "mixed"),         # a round and a rest, ragged edges
    (8200, 1504, 4112, 16, 40, "each"),         # chains of tiles, most with many adapters
    (8200, 1504, 4112, 8, 4200, "each"),        # the same, rows as they are
    (8200, 1536, 4112, 40, 2, -1),              # no row with an adapter
    (65600, 32, 14336, 8, 3, "mixed"),          # chains of tiles of one step, rows as they are
    (33000, 96, 14336, 24, 5, "mixed"),         # of two
    (33000, 160, 14336, 16, 4, "pairs"),        # of three
]
# (counts, N, K) of the layer: the data gradient sums over N
GRADS = [
    ([4090], 2064, 4096), ([5200, 0, 3000], 2064, 4128), ([1, 4000, 0, 255, 257, 4200], 2080, 4096),
    ([50000, 5, 0, 50002], 16, 8192), ([30000, 129, 40001], 80, 8192), ([100, 40001], 144, 8224),
    ([30001], 192, 8192),
]
# down projections of rows as they are, too many rows times ranks for spread dots: (M, K, N, r, L, ids)
UNSORTED = [
    (200, 288, 528, 512, 30, "each"), (200, 288, 528, 512, 30, "pairs"), (200, 288, 528, 512, 30, 7),
    (333, 544, 1040, 200, 200, "mixed"), (65600, 32, 16, 8, 40, "mixed"), (65600, 96, 16, 24, 40, "each"),
    (65600, 64, 32, 24, 3, "pairs"),
]


def make(M, K, N, r, L, ids, dev):
    g = torch.Generator(device=dev).manual_seed(M + K + N)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)
    x = rnd(M, K)
    x = torch.where(torch.rand((M, K), generator=g, device=dev) < 0.01, 20 * x, x).bfloat16()
    w, a, b = (rnd(N, K) * 0.05).bfloat16(), (rnd(L, r, K) * K ** -0.5).bfloat16(), (rnd(L, N, r) * 0.3).bfloat16()
    h = torch.Generator().manual_seed(M)
    pick = lambda lo, hi: int(torch.randint(lo, hi, (), generator=h))
    if ids == "mixed":
        out = []
        while len(out) < M:
            out += [pick(-1, L + 1)] * (pick(0, 6) ** 3 + 1)
        ids = out[:M]
    elif ids == "pairs":
        out = []
        while len(out) < M:
            two = [pick(-1, L), pick(0, L)]
            out += [two[pick(0, 2)] for _ in range(100)]
        ids = out[:M]
    elif ids == "each":
        ids = torch.randint(-1, L, (M,), generator=h).tolist()
    else:
        ids = [ids] * M
    return x, w, a, b, torch.tensor(ids, dtype=torch.int32, device=dev), 3 * torch.rand(L, generator=g, device=dev) - 1


def within(got, ref, bound):
    over = (got.double() - ref).abs_().sub_(bound)
    assert over.isfinite().all() and (over <= 0).all(), float(over.max())


def check(y, x, w, a, b, ids, s):
    K, r = x.shape[1], a.shape[1]
    x, w = x.double(), w.double()
    ref, S = x @ w.t(), x.abs() @ w.abs().t()
    err = S * ((K + 2) * N23)
    for l in ids.unique().tolist():
        if not 0 <= l < a.shape[0]:
            continue
        rows = (ids == l).nonzero().flatten()
        al, bl, sl = a[l].double(), b[l].double(), s[l].double()
        ref[rows] += sl * ((x[rows] @ al.t()) @ bl.t())
        low = sl.abs() * ((x[rows].abs() @ al.abs().t()) @ bl.abs().t())
        err[rows] += ((K + 4) * N23 + 2.0 ** -16) * low
        S[rows] += low
    err += (2 * r + 4) * N23 * S
    within(y, ref, H * ref.abs() + (1 + H) * err)


def call(x, w, a, b, ids, s):
    """Through the C entry, every byte of scratch a NaN, y at the front of a longer buffer."""
    (M, K), N, (L, r) = x.shape, w.shape[0], a.shape[:2]
    nws = gm.lib().lora_linear_ws_bytes(M, N, K, L, r)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=x.device)
    y = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device=x.device)
    st = gm.lib().lora_linear_fwd(x.data_ptr(), M, K, w.data_ptr(), N, a.data_ptr(), b.data_ptr(), L, r,
                                  ids.data_ptr(), s.data_ptr(), y.data_ptr(), ws.data_ptr(), nws,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0, gm.last_error()
    assert (y[M:] == 7).all()
    return y[:M]


@pytest.mark.parametrize("M,K,N,r,L,ids", FORWARD + UNSORTED)
def test_adapter_linear(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, dev)
    y = call(x, w, a, b, ids, s)
    check(y, x, w, a, b, ids, s)
    assert torch.equal(y, gm.lora_linear_fwd(x, w, a, b, ids, scale=s))     # one order of the sums


@pytest.mark.parametrize("M,K,N,r,L,ids", [FORWARD[1], FORWARD[3], UNSORTED[0], UNSORTED[1], UNSORTED[5]])
def test_what_is_not_finite_stays_in_its_rows(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, dev)
    ids[0], ids[1], ids[2] = 0, 1, -1
    clean = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    b[1, 5, :], b[1, N - 1, 2], a[1, 1, 7] = float("nan"), float("inf"), float("-inf")
    x[2, 9] = float("nan")
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    hit = ids == 1
    hit[2] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert y[2].isnan().all() and y[1, 5].isnan()


@pytest.mark.parametrize("M,K,N,r,L,ids", FORWARD[1:3])
def test_a_sorted_row_is_the_same_wherever_it_stands(dev, M, K, N, r, L, ids):
    x, w, a, b, ids, s = make(M, K, N, r, L, ids, dev)
    y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s)
    p = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(dev)
    assert torch.equal(gm.lora_linear_fwd(x[p], w, a, b, ids[p], scale=s), y[p])


def test_captured_and_replayed(dev):
    x, w, a, b, ids, s = make(*FORWARD[1], dev)
    ws = torch.empty(gm.lib().lora_linear_ws_bytes(x.shape[0], w.shape[0], x.shape[1], *a.shape[:2]),
                     dtype=torch.uint8, device=dev)
    gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gm.lora_linear_fwd(x, w, a, b, ids, scale=s, ws=ws)
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        ids.copy_(torch.randint(-1, a.shape[0], ids.shape, generator=g).int())
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, gm.lora_linear_fwd(x, w, a, b, ids, scale=s))


def make_grads(counts, N, K, scaled, dev):
    g = torch.Generator(device=dev).manual_seed(N + K)
    off = torch.tensor([0] + counts).cumsum(0)
    M, E = int(off[-1]), len(counts)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)
    x = rnd(M, K)
    x = torch.where(torch.rand((M, K), generator=g, device=dev) < 0.01, 20 * x, x).bfloat16()
    r = torch.rand(M, generator=g, device=dev) - 0.25 if scaled else None
    return rnd(M, N).bfloat16(), x, (rnd(E, N, K) * 0.05).bfloat16(), off.tolist(), off.to(dev), r


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("counts,N,K", GRADS)
def test_gradients(dev, counts, N, K, scaled):
    dy, x, w, off, offd, r = make_grads(counts, N, K, scaled, dev)
    M, E = x.shape[0], len(counts)
    L, nws = gm.lib(), gm.lib().grouped_linear_bwd_ws_bytes(E, M, N, K, scaled)
    ws = torch.full((nws,), 255, dtype=torch.uint8, device=dev)
    dx = torch.full((M + 300, K), 7.0, dtype=torch.bfloat16, device=dev)
    dr = torch.full((M + 300,), 7.0, device=dev)
    st = L.grouped_linear_bwd(dy.data_ptr(), x.data_ptr(), offd.data_ptr(), E, M, w.data_ptr(), N, K,
                              r.data_ptr() if scaled else 0, dx.data_ptr(), dr.data_ptr() if scaled else 0, 0, 0,
                              ws.data_ptr(), nws, torch.cuda.current_stream().cuda_stream)
    assert st == 0, gm.last_error()
    assert (dx[M:] == 7).all() and (dr[M if scaled else 0:] == 7).all()
    dx2, dw, dr2 = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r, dw_dtype=torch.float32)
    assert torch.equal(dx[:M], dx2) and (not scaled or torch.equal(dr[:M], dr2))
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        d, xe, we = dy[rows].double(), x[rows].double(), w[e].double()
        ref, mag = d @ we, d.abs() @ we.abs()
        n = off[e + 1] - off[e]
        if scaled:
            re = r[rows].double()[:, None]
            within(dr[rows], (ref * xe).sum(1), (N + K + 4) * N23 * (mag * xe.abs()).sum(1))
            ref, mag, d = ref * re, mag * re.abs(), d * re
        within(dx[rows], ref, H * ref.abs() + (1 + H) * (N + 2) * N23 * mag)
        mag = d.abs().t() @ xe.abs()
        bound = (n + 2) * N23 * mag
        if scaled:
            bound = (1 + 2.0 ** -7) * bound + (H + 2.0 ** -20) * mag
        within(dw[e], d.t() @ xe, bound)


@pytest.mark.parametrize("counts,N,K", [GRADS[1], GRADS[4]])
def test_gradients_keep_what_is_not_finite(dev, counts, N, K):
    dy, x, w, off, offd, r = make_grads(counts, N, K, True, dev)
    clean = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    last = off[-2]                                  # the last expert's first row
    dy[1, 3], x[1, 7], w[-1, N - 1, K - 1] = float("nan"), float("inf"), float("-inf")
    dx, dw, dr = gm.grouped_linear_bwd(dy, x, offd, w, row_scale=r)
    fine = torch.ones(x.shape[0], dtype=torch.bool, device=dev)
    fine[1] = False
    fine[last:] = False
    assert torch.equal(dx[fine], clean[0][fine]) and torch.equal(dr[fine], clean[2][fine])
    assert dx[1].isnan().all() and torch.equal(dx[last:, :K - 1], clean[0][last:, :K - 1])
    assert torch.equal(dw[1:], clean[1][1:]) and dw[0, 3].isnan().all()
