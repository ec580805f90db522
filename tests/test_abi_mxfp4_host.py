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
