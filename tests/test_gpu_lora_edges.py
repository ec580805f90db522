"""The adapter linear on the GPU at the edges of its range, against FP64 (bounds:
oracle/bf16_oracle.py)."""
import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import bf16_oracle as B

pytestmark = pytest.mark.gpu


def to64(t):
    return t.double().cpu().numpy()


# one launch, dots and MFMA blocks of few rows, the join, tiles of unsorted and of sorted rows,
# down projections in tiles
@pytest.mark.parametrize("M,K,N,r,L,runs", [
    (2, 64, 48, 16, 2, 1), (5, 64, 48, 16, 3, 1), (16, 64, 48, 16, 2, 8), (40, 4096, 272, 8, 9, 1),
    (100, 64, 272, 16, 60, 1), (300, 64, 272, 16, 4, 1), (1030, 96, 48, 160, 3, 40)])
def test_low_rank_values_past_the_largest_bf16(dev, M, K, N, r, L, runs):
    """a x of 1.998 * 2^127, finite in fp32 and next to 2^128 in bf16: b brings it back into
    range, so the result is finite."""
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g)
    x[:, :2] = 2.0 ** 64
    w = torch.randn((N, K), generator=g) * 0.05
    w[:, :2] = 0
    a = torch.randn((L, r, K), generator=g)
    a[:, :, 0], a[:, :, 1] = 1.9921875 * 2.0 ** 63, 0.75 * 2.0 ** 56
    a[:, ::2] *= -1
    b = torch.randn((L, N, r), generator=g) * 2.0 ** -125
    x, w, a, b = (t.bfloat16() for t in (x, w, a, b))
    ids = torch.randint(-1, L, (M,), generator=g).int()[torch.arange(M) // runs]
    ids[0] = 0
    y = gm.lora_linear_fwd(x.to(dev), w.to(dev), a.to(dev), b.to(dev), ids.to(dev))
    torch.cuda.synchronize()
    args = [to64(t) for t in (x, w, a, b)] + [ids.numpy()]
    err = np.abs(to64(y) - B.lora_fwd(*args))
    assert np.isfinite(err).all() and (err <= B.lora_bound(*args)).all()


@pytest.mark.parametrize("r", [8, 16, 24, 40])
def test_adapters_of_other_ranks_trained_with_zeros(dev, r):
    """Ranks that are no multiple of 32, padded with zeros to one: gradients are those of the
    rank itself, the padding's are zeros, and the padded weights serve as the others do.
    Gradients in fp32 of exact products of bf16 values: n terms are off by n 2^-23 of their
    magnitudes; h and dh are rounded to bf16 for both sides."""
    g = torch.Generator().manual_seed(r)
    M, K, N, L, pad = 240, 256, 288, 4, -(-r // 32) * 32
    rnd = lambda *s: torch.randn(s, generator=g)
    x, w = rnd(M, K).bfloat16().to(dev), (0.05 * rnd(N, K)).bfloat16().to(dev)
    a, b = torch.zeros((L, pad, K)), torch.zeros((L, N, pad))
    a[:, :r], b[:, :, :r] = rnd(L, r, K) * K ** -0.5, rnd(L, N, r) * 0.3
    a, b = a.bfloat16().to(dev), b.bfloat16().to(dev)
    ids = torch.randint(-1, L, (M,), generator=g).int().to(dev)
    off, _, tok_of, _ = gm.route_plan(ids.view(M, 1), L)
    n = int(off[-1])
    xs = x[tok_of[:n].long()].contiguous()
    dz = rnd(n, N).bfloat16().to(dev)
    h = gm.grouped_linear_fwd(xs, off, a)
    dh, db, _ = gm.grouped_linear_bwd(dz, h, off, b, dw_dtype=torch.float32)
    _, da, _ = gm.grouped_linear_bwd(dh, xs, off, a, dw_dtype=torch.float32, need_dx=False)
    y = gm.lora_linear_fwd(x, w, a, b, ids)
    torch.cuda.synchronize()
    for t in (h[:, r:], dh[:, r:], da[:, r:], db[:, :, r:]):
        assert not t.any()
    o, z, hh, d, xx = off.cpu().numpy(), to64(dz), to64(h[:, :r]), to64(dh[:, :r]), to64(xs)
    a64, b64, w64 = to64(a[:, :r]), to64(b[:, :, :r]), to64(w)
    for got, dy, v, wt in ((db[:, :, :r], z, hh, b64), (da[:, :r], d, xx, a64)):
        ref, mag = B.linear_bwd(dy, v, wt, o)[1], B.linear_bwd(np.abs(dy), np.abs(v), np.abs(wt), o)[1]
        assert (np.abs(to64(got) - ref) <= (n + 2) * 2.0 ** -23 * mag).all()
    ref, mag = B.linear_bwd(z, hh, b64, o)[0], B.linear_bwd(np.abs(z), np.abs(hh), np.abs(b64), o)[0]
    assert (np.abs(d - ref) <= 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * (N + 2) * 2.0 ** -23 * mag).all()
    args = (to64(x), w64, a64, b64, ids.cpu().numpy())
    assert (np.abs(to64(y) - B.lora_fwd(*args)) <= B.lora_bound(*args)).all()


@pytest.mark.parametrize("M,L", [(40, 5), (200, 90), (12, 12)])
def test_unsorted_rows_are_right_in_any_order(dev, M, L):
    """Rows as they are, in four orders: dots or MFMA blocks go by the adapters among sixteen
    rows, so a row's last bits may differ, within the bounds, and the same call repeats itself."""
    g = torch.Generator().manual_seed(M)
    K, N, r = 544, 272, 16
    rnd = lambda *s: torch.randn(s, generator=g)
    x, w = rnd(M, K).bfloat16(), (0.05 * rnd(N, K)).bfloat16()
    a, b = (rnd(L, r, K) * K ** -0.5).bfloat16(), (0.3 * rnd(L, N, r)).bfloat16()
    ids = torch.randint(-1, L, (M,), generator=g).int()
    args = [to64(t) for t in (x, w, a, b)] + [ids.numpy()]
    ref, bound = B.lora_fwd(*args), B.lora_bound(*args)
    for p in (torch.arange(M), ids.argsort(), torch.randperm(M, generator=g), torch.randperm(M, generator=g)):
        call = [t.to(dev) for t in (x[p], w, a, b, ids[p])]
        y = gm.lora_linear_fwd(*call)
        assert torch.equal(y, gm.lora_linear_fwd(*call))
        assert (np.abs(to64(y) - ref[p]) <= bound[p]).all()
