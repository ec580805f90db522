"""Refusals of grouped_linear_bwd and lora_linear_fwd, on the host (no kernel is
launched)."""
import ctypes

import pytest
import torch

import grouped_gemm_mxfp8_amd as gm

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(0x7f0000001000)        # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x7f0000001008)
BIG = 1 << 60

BWD = dict(dy=P, x=P, off=P, E=2, M=64, w=P, N=64, K=64, r=P, dx=P, dr=P, dw=P, flags=0, ws=P, n=BIG)
LORA = dict(x=P, M=8, K=64, w=P, N=64, a=P, b=P, L=2, r=16, ids=P, s=P, y=P, ws=P, n=BIG)


@pytest.mark.parametrize("change,status,text", [
    (dict(dy=None), INVALID, "NULL"), (dict(x=None), INVALID, "NULL"), (dict(off=None), INVALID, "NULL"),
    (dict(w=None), INVALID, "NULL"), (dict(ws=None), INVALID, "NULL"),
    (dict(dx=None, dr=None, dw=None), INVALID, "neither"),
    (dict(dx=None), INVALID, "dr needs"), (dict(r=None), INVALID, "dr needs"),
    (dict(E=0), INVALID, "sizes"), (dict(E=1025), INVALID, "sizes"), (dict(M=-1), INVALID, "sizes"),
    (dict(N=0), INVALID, "sizes"), (dict(K=0), INVALID, "sizes"),
    (dict(K=48), UNSUPPORTED, "K % 32"), (dict(N=24), UNSUPPORTED, "N % 16"),
    (dict(K=(1 << 21) + 32), UNSUPPORTED, "2^21"), (dict(N=(1 << 21) + 16), UNSUPPORTED, "2^21"),
    (dict(M=1 << 31), UNSUPPORTED, "2^31"),
    (dict(M=(1 << 31) - 1, N=1 << 21, K=1 << 21), UNSUPPORTED, "launch"),
    (dict(flags=4), INVALID, "flags"), (dict(flags=2), INVALID, "fp32 dw"),
    (dict(dy=ODD), INVALID, "aligned"), (dict(x=ODD), INVALID, "aligned"), (dict(w=ODD), INVALID, "aligned"),
    (dict(dx=ODD), INVALID, "aligned"), (dict(dw=ODD), INVALID, "aligned"), (dict(ws=ODD), INVALID, "aligned"),
    (dict(n=16), WORKSPACE, "needs"),
])
def test_linear_bwd_refusals(mxlib, change, status, text):
    assert mxlib.grouped_linear_bwd(*{**BWD, **change}.values(), None) == status
    assert text in mxlib.mx_last_error().decode()


@pytest.mark.parametrize("change,status,text", [
    (dict(x=None), INVALID, "NULL"), (dict(w=None), INVALID, "NULL"), (dict(a=None), INVALID, "NULL"),
    (dict(b=None), INVALID, "NULL"), (dict(ids=None), INVALID, "NULL"), (dict(y=None), INVALID, "NULL"),
    (dict(ws=None), INVALID, "NULL"),
    (dict(M=-1), INVALID, "sizes"), (dict(L=0), INVALID, "sizes"), (dict(r=0), INVALID, "sizes"),
    (dict(N=0), INVALID, "sizes"), (dict(K=0), INVALID, "sizes"),
    (dict(K=48), UNSUPPORTED, "K % 32"), (dict(N=24), UNSUPPORTED, "N % 16"), (dict(r=12), UNSUPPORTED, "r % 8"),
    (dict(r=520), UNSUPPORTED, "512"), (dict(K=(1 << 21) + 32), UNSUPPORTED, "2^21"),
    (dict(N=(1 << 21) + 16), UNSUPPORTED, "2^21"), (dict(M=1 << 31), UNSUPPORTED, "2^31"),
    (dict(M=(1 << 31) - 1, N=1 << 21), UNSUPPORTED, "launch"),
    (dict(x=ODD), INVALID, "aligned"), (dict(w=ODD), INVALID, "aligned"), (dict(a=ODD), INVALID, "aligned"),
    (dict(b=ODD), INVALID, "aligned"), (dict(y=ODD), INVALID, "aligned"), (dict(ws=ODD), INVALID, "aligned"),
    (dict(n=16), WORKSPACE, "needs"), (dict(n=256, M=2, r=24), WORKSPACE, "needs"),
    (dict(ws=None, M=2, r=24), INVALID, "NULL ws"),
])
def test_lora_refusals(mxlib, change, status, text):
    assert mxlib.lora_linear_fwd(*{**LORA, **change}.values(), None) == status
    assert text in mxlib.mx_last_error().decode()


def test_workspace_sizes(mxlib):
    for L in (mxlib,):
        assert L.grouped_linear_bwd_ws_bytes(2, 0, 16, 32, 0) == 256
        assert L.grouped_linear_bwd_ws_bytes(2, 8, 24, 32, 1) == 0
        assert L.lora_linear_ws_bytes(0, 16, 32, 1, 8) == 256
        assert L.lora_linear_ws_bytes(1, 16, 32, 1, 9) == 0
    # 256 stands for no scratch at all, also where all of it would fit into 256 bytes
    assert mxlib.lora_linear_ws_bytes(2, 16, 96, 2, 24) == 512
    assert mxlib.lora_linear_ws_bytes(1, 4096, 4096, 8, 16) == 256
    # no rows: nothing to launch for an adapter linear
    assert mxlib.lora_linear_fwd(None, 0, 64, None, 64, None, None, 1, 8, None, None, None, None, 0, None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(TypeError):
        gm.grouped_linear_bwd(torch.zeros((4, 16)), bf(4, 32), off, bf(1, 16, 32))
    with pytest.raises(ValueError, match="GPU"):
        gm.grouped_linear_bwd(bf(4, 16), bf(4, 32), off, bf(1, 16, 32))
    with pytest.raises(TypeError):
        gm.lora_linear_fwd(torch.zeros((4, 32)), bf(16, 32), bf(1, 8, 32), bf(1, 16, 8), off.int())
    with pytest.raises(ValueError, match="GPU"):
        gm.lora_linear_fwd(bf(4, 32), bf(16, 32), bf(1, 8, 32), bf(1, 16, 8), torch.zeros(4, dtype=torch.int32))
