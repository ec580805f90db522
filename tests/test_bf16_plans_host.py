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


@pytest.mark.parametrize("form,G,M,N,K,kind", [
    # 1024 middle tiles of two steps, and 2048 small ones
    (FORWARD, 1, 4096, 4096, 128, MIDDLE), (DATA_GRAD, 1, 4096, 4096, 16, MIDDLE),
    # as many of three; fewer than a GPU has room for: small ones
    (FORWARD, 1, 8192, 2048, 192, MIDDLE), (FORWARD, 1, 300, 2048, 64, SMALL), (DATA_GRAD, 4, 512, 128, 64, SMALL),
    # more than 1024 middle tiles, more than 1024 small tiles of few rows each
    (DATA_GRAD, 4, 52000, 32, 16, MIDDLE), (DATA_GRAD, 28, 96, 2080, 128, SMALL), (DATA_GRAD, 9, 5, 12992, 64, SMALL),
])
def test_short_sums_take_the_faster_tiles_too(plan, form, G, M, N, K, kind):
    """Sums of up to three steps: no shares of K, and both kinds of tiles are considered."""
    assert plan(form, G, M, M, N, K, 8) == (kind, 1)
