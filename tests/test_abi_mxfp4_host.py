"""Refusals of the MXFP4 entry points, on the host (no kernel is launched)."""
import ctypes

import pytest
import torch

import grouped_gemm_mxfp8_amd as gm

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(0x7f0000001000)        # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x7f0000001008)


def err(L):
    return L.mx_last_error().decode()


@pytest.mark.parametrize("args,status,text", [
    ((None, 1, 64, 64, P, P, None, None), INVALID, "NULL"),
    ((P, 0, 64, 64, P, P, None, None), INVALID, "sizes"),
    ((P, 1, -1, 64, P, P, None, None), INVALID, "sizes"),
    ((P, 1, 64, 48, P, P, None, None), UNSUPPORTED, "multiple of 32"),
    ((P, 1, 64, 64, P, None, None, None), INVALID, "go together"),
    ((P, 1, 64, 64, None, None, None, P), INVALID, "go together"),
    ((P, 1, 64, 64, None, None, None, None), INVALID, "no output"),
    ((P, 1, 48, 64, None, None, P, P), UNSUPPORTED, "R % 32"),
    ((ODD, 1, 64, 64, P, P, None, None), INVALID, "aligned"),
    ((P, 1, 64, 64, ODD, P, None, None), INVALID, "aligned"),
    ((P, 1 << 20, 64, 64, None, None, P, P), UNSUPPORTED, "too large"),
    ((P, 1 << 40, 1 << 40, 64, P, P, None, None), UNSUPPORTED, "too large"),
    ((P, 1, 1 << 62, 1 << 62, P, P, None, None), UNSUPPORTED, "too large"),
])
def test_quantize_refusals(mxlib, args, status, text):
    assert mxlib.mxfp4_quantize(*args, None) == status
    assert text in err(mxlib)


@pytest.mark.parametrize("args,status,text", [
    ((None, P, 4, 64, P), INVALID, "NULL"),
    ((P, None, 4, 64, P), INVALID, "NULL"),
    ((P, P, 4, 64, None), INVALID, "NULL"),
    ((P, P, -4, 64, P), INVALID, "sizes"),
    ((P, P, 4, 40, P), UNSUPPORTED, "multiple of 32"),
    ((ODD, P, 4, 64, P), INVALID, "aligned"),
    ((P, P, 1 << 50, 64, P), UNSUPPORTED, "too large"),
])
def test_dequantize_refusals(mxlib, args, status, text):
    assert mxlib.mxfp4_dequantize(*args, None) == status
    assert text in err(mxlib)


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(TypeError):
        gm.mxfp4_quantize(torch.zeros((4, 32)))
    with pytest.raises(ValueError, match="GPU"):
        gm.mxfp4_quantize(torch.zeros((4, 32), dtype=torch.bfloat16))
    q = gm.Mx4Tensor(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.uint8))
    with pytest.raises(ValueError, match="GPU"):
        gm.mxfp4_dequantize(q)


FP4, FP8FP4, BF16, FP8 = gm.MX_DTYPE_MXFP4, gm.MX_DTYPE_MXFP8_MXFP4, gm.MX_DTYPE_BF16, gm.MX_DTYPE_MXFP8


@pytest.mark.parametrize("dtype", [FP4, FP8FP4])
@pytest.mark.parametrize("change,status,text", [
    (dict(x=None), INVALID, "NULL"),
    (dict(y=None), INVALID, "NULL"),
    (dict(xs=None), INVALID, "scales"),
    (dict(ws=None), INVALID, "scales"),
    (dict(K=48), UNSUPPORTED, "K % 32"),
    (dict(N=40), UNSUPPORTED, "N % 32"),
    (dict(N=1 << 32), UNSUPPORTED, "up to 2^26"),
    (dict(K=1 << 32), UNSUPPORTED, "up to 2^26"),
    (dict(N=(1 << 26) + 32), UNSUPPORTED, "up to 2^26"),
    (dict(K=(1 << 26) + 32), UNSUPPORTED, "up to 2^26"),
    (dict(E=0), INVALID, "sizes"),
    (dict(E=1025), INVALID, "sizes"),
    (dict(M=-1), INVALID, "sizes"),
    (dict(w=ODD), INVALID, "aligned"),
    (dict(y=ODD), INVALID, "aligned"),
    (dict(xs=ctypes.c_void_p(0x7f0000001002)), INVALID, "aligned"),
])
def test_linear_refusals(mxlib, dtype, change, status, text):
    a = dict(x=P, xs=P, off=P, E=4, M=8, w=P, ws=P, N=64, K=64, r=None, y=P)
    a.update(change)
    assert mxlib.grouped_linear_fwd(dtype, *a.values(), None) == status
    assert text in err(mxlib)


def test_linear_unknown_dtype(mxlib):
    for dtype in (-1, 4):
        assert mxlib.grouped_linear_fwd(dtype, P, P, P, 4, 8, P, P, 64, 64, None, P, None) == INVALID
        assert "dtype" in err(mxlib)


@pytest.mark.parametrize("change,status,text", [
    (dict(dtype=FP8FP4), INVALID, "dtype"),
    (dict(T=-1), INVALID, "sizes"),
    (dict(k=0), INVALID, "sizes"),
    (dict(k=9), INVALID, "sizes"),
    (dict(E=0), INVALID, "sizes"),
    (dict(T=129), UNSUPPORTED, "tokens"),
    (dict(E=1025), UNSUPPORTED, "experts"),
    (dict(E=100, k=65), UNSUPPORTED, "slots"),
    (dict(H=192), UNSUPPORTED, "multiples"),
    (dict(F=96), UNSUPPORTED, "multiples"),
    (dict(F=1 << 25), UNSUPPORTED, "multiples"),
    (dict(x=None), INVALID, "NULL"),
    (dict(logits=None), INVALID, "NULL"),
    (dict(ws=None), INVALID, "NULL"),
    (dict(s1=None), INVALID, "scales"),
    (dict(dtype=BF16), INVALID, "scales"),
    (dict(x=ODD), INVALID, "aligned"),
    (dict(out=ODD), INVALID, "aligned"),
    (dict(s2=ctypes.c_void_p(0x7f0000001001)), INVALID, "aligned"),
    (dict(ws=ctypes.c_void_p(0x7f0000001010)), INVALID, "256-byte"),
    (dict(n=100), WORKSPACE, "needs"),
])
def test_layer_refusals(mxlib, change, status, text):
    a = dict(dtype=FP4, x=P, logits=P, T=4, E=8, k=2, H=256, F=256, w1=P, s1=P, w2=P, s2=P, out=P,
             ws=P, n=1 << 30)
    a.update(change)
    assert mxlib.moe_layer_fwd(*a.values(), None) == status
    assert text in err(mxlib)


def test_layer_workspace_bytes(mxlib):
    f = mxlib.moe_layer_ws_bytes
    T, E, k, H, F = 64, 64, 8, 2048, 1408
    need = T * H * 33 // 32 + T * k * F * 33 // 32 + T * k * 8 + E * 16
    parts = 8 * T * H * 4          # at most eight partial sums of the output
    assert need <= f(FP4, T, E, k, H, F) <= need + parts + 16 * 256
    assert f(FP4, T, E, k, H, F) == f(FP8, T, E, k, H, F)
    assert T * k * F * 2 <= f(BF16, T, E, k, H, F)
    assert f(FP4, 0, E, k, H, F) > 0
    assert f(FP4, 129, E, k, H, F) == 0 and f(FP8FP4, T, E, k, H, F) == 0
    # the largest sizes do not overflow
    assert f(BF16, 128, 1024, 64, 1 << 24, 1 << 24) > 128 * 64 * (1 << 25)


@pytest.mark.parametrize("batch,R,C", [
    (1, 1 << 32, 32), (1, 1 << 20, 1 << 17), (1 << 15, 1 << 17, 32),
    (1, (1 << 32) - 128, 32),              # 2^37 - 4096: one workgroup more than fit
    (1, 1 << 38, 32), (3, 1 << 30, 1 << 10),
])
def test_sizes_past_what_a_launch_takes_are_refused(mxlib, batch, R, C):
    """A launch holds fewer than 2^32 threads, which take 32 values each, 256 of
    them a workgroup: larger tensors are refused, not left to the launch."""
    for args in ((P, P, None, None), (None, None, P, P), (P, P, P, P)):
        assert mxlib.mxfp4_quantize(P, batch, R, C, *args, None) == UNSUPPORTED
        assert "too large" in err(mxlib)
    assert mxlib.mxfp4_dequantize(P, P, batch * R, C, P, None) == UNSUPPORTED
    assert "too large" in err(mxlib)
