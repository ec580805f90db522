"""Which kernel the bf16 products take (asked of the library's planner; no GPU needed): the
cases written for the large tiles and for unsorted down projections have to reach them."""
import ctypes

import pytest

from tests import test_gpu_bf16_large as T

LARGE, SMALL, MIDDLE = 0, 1, 2
FORWARD, DATA_GRAD, WEIGHT_GRAD = 0, 1, 2


@pytest.fixture(scope="module")
def plan(mxlib):
    """(kernel, shares of K) of a product."""
    f, n = mxlib.mx_internal_bf16_plan, ctypes.c_int64
    f.restype, f.argtypes = ctypes.c_int32, [ctypes.c_int32] * 2 + [n] * 4 + [ctypes.c_int32]
    return lambda form, G, rows, M, N, K, r=0: divmod(f(form, G, rows, M, N, K, r), 4)[::-1]


def unsorted(mxlib, M, K, N, r, L):
    """Whether rows stay as they are: scratch for h alone (no split of K)."""
    return mxlib.lora_linear_ws_bytes(M, N, K, L, r) == 256 + (4 * M * r + 255) // 256 * 256


@pytest.mark.parametrize("M,K,N,r,L,ids", T.FORWARD)
def test_adapter_linear_reaches_the_large_tiles(plan, M, K, N, r, L, ids):
    assert plan(FORWARD, 1, M, M, N, K, r) == (LARGE, 1)


def test_adapter_linear_in_every_order_and_rest(mxlib):
    order = {unsorted(mxlib, M, K, N, r, L) for M, K, N, r, L, _ in T.FORWARD}
    tiles = [-(-M // 256) * -(-N // 256) for M, K, N, r, L, _ in T.FORWARD]
    assert order == {False, True}
    # a whole round alone, a rest left to the middle tiles, chains
    assert 256 in tiles and any(256 < t <= 256 + 176 for t in tiles) and max(tiles) >= 512
    assert {-(-K // 64) for _, K, *_ in T.FORWARD} >= {1, 2, 3}


@pytest.mark.parametrize("counts,N,K", T.GRADS)
def test_data_gradient_reaches_the_large_tiles(plan, counts, N, K):
    M = sum(counts)
    assert plan(DATA_GRAD, len(counts), M, M, K, N) == (LARGE, 1)


@pytest.mark.parametrize("M,K,N,r,L,ids", T.UNSORTED)
def test_down_projection_stays_unsorted_and_unspread(plan, mxlib, M, K, N, r, L, ids):
    assert plan(FORWARD, 1, M, M, N, K, r)[1] == 1 and unsorted(mxlib, M, K, N, r, L) and M * r > 65536
