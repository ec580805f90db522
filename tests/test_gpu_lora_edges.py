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
