"""MXFP4 quantizer and dequantizer on the GPU: codes, scales and values
bit-exact against the FP64 oracle."""
import numpy as np
import pytest
import torch

import grouped_gemm_mxfp8_amd as gm
from oracle import mx4_oracle as P

pytestmark = pytest.mark.gpu


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


def bits(a):
    return torch.from_numpy(np.asarray(a, np.uint16).view(np.int16)).view(torch.bfloat16)


def check(x, dev, rowwise=True, colwise=False):
    q = gm.mxfp4_quantize(x.to(dev), rowwise=rowwise, colwise=colwise)
    torch.cuda.synchronize()
    for name, ref in (("row", to64(x)), ("col", np.swapaxes(to64(x), -1, -2))):
        if name in q:
            codes, scales = P.quantize4_lastdim(ref)
            assert np.array_equal(q[name].codes.cpu().numpy(), codes), name
            assert np.array_equal(q[name].scales.cpu().numpy(), scales), name
    return q


def every_pattern(seed):
    """Every bf16 pattern with a finite value, in shuffled blocks, alone and
    next to a large, a unit and a tiny value."""
    rng = np.random.default_rng(seed)
    b = np.arange(1 << 16)
    b = b[(b >> 7 & 255) != 255]
    parts = []
    for anchor in (None, 0x4380, 0x3f80, 0x0100, 0x7f7f, 0x0001):
        p = rng.permutation(b)
        p = p[:len(p) // 32 * 32].reshape(-1, 32).copy()
        if anchor is not None:
            p[:, 0] = anchor
        parts.append(p)
        # blocks of nearly equal magnitudes: every rounding border is met
        s = np.sort(b).reshape(-1)[:len(b) // 32 * 32].reshape(-1, 32)
        parts.append(s)
    return bits(np.concatenate(parts))


def test_every_bf16_pattern_row_and_col(dev):
    x = every_pattern(0)
    R = x.shape[0] // 32 * 32
    check(x, dev)
    check(x[:R].contiguous(), dev, rowwise=False, colwise=True)
    check(x[:R].t().contiguous(), dev, rowwise=False, colwise=True)


@pytest.mark.parametrize("shape", [(1, 32), (1, 4096), (3, 96), (1003, 1408), (257, 2048),
                                   (2, 5, 64), (7, 33, 160)])
def test_rows(dev, shape):
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(shape, generator=g) * torch.exp(4 * torch.randn(shape, generator=g))).bfloat16()
    check(x, dev)


@pytest.mark.parametrize("shape", [(32, 32), (256, 64), (288, 96), (1408, 2048), (3, 64, 32),
                                   (5, 544, 160)])
def test_columns(dev, shape):
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(shape, generator=g) * torch.exp(4 * torch.randn(shape, generator=g))).bfloat16()
    check(x, dev, rowwise=True, colwise=True)


def test_zero_rows_and_nonfinite_blocks(dev):
    x = torch.randn((64, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    x[0] = 0
    x[1] = -0.0
    x[2, 5], x[3, 40], x[4, 100] = float("inf"), float("-inf"), float("nan")
    q = check(x, dev, colwise=True)
    v = gm.mxfp4_dequantize(q["row"]).float().cpu()
    assert torch.isnan(v[2, :32]).all() and not torch.isnan(v[2, 32:]).any()
    assert torch.isnan(v[3, 32:64]).all() and torch.isnan(v[4, 96:]).all()
    assert not v[0].any() and torch.signbit(v[1]).all()


def test_dequantize_every_code_and_scale(dev):
    """All 256 code bytes under all 256 scales."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 16, 16).expand(256, -1, -1).contiguous()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1, 1).expand(-1, 16, 1).contiguous()
    y = gm.mxfp4_dequantize(gm.Mx4Tensor(codes.to(dev), scales.to(dev)))
    ref = P.dequantize4_lastdim(codes.numpy(), scales.numpy())
    got = to64(y)
    # 6 * 2^126 and 4 * 2^126 (2^127: 2 and more) pass the largest finite bf16
    big = np.abs(ref) > float(torch.finfo(torch.bfloat16).max)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fine = ~big & ~np.isnan(ref)
    assert np.array_equal(got[fine], ref[fine])
    assert np.array_equal(np.signbit(got[fine]), np.signbit(ref[fine]))
    assert np.isinf(got[big]).all()


def test_round_trip_on_another_stream_and_in_a_graph(dev):
    x = torch.randn((300, 512), generator=torch.Generator().manual_seed(1)).bfloat16().to(dev)
    want = gm.mxfp4_dequantize(gm.mxfp4_quantize(x)["row"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = gm.mxfp4_dequantize(gm.mxfp4_quantize(x)["row"])
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gm.mxfp4_dequantize(gm.mxfp4_quantize(x)["row"])
    for seed in (2, 3, 4):
        x.copy_(torch.randn((300, 512), generator=torch.Generator().manual_seed(seed)).bfloat16())
        g.replay()
        want = gm.mxfp4_dequantize(gm.mxfp4_quantize(x)["row"])
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_tensors(dev):
    q = gm.mxfp4_quantize(torch.empty((0, 64), dtype=torch.bfloat16, device=dev))
    assert q["row"].codes.shape == (0, 32) and q["row"].scales.shape == (0, 2)
    assert gm.mxfp4_dequantize(q["row"]).shape == (0, 64)
