"""moe_unpermute_combine_bwd's output rows may not lie over the rows it reads: tokens are
read while others' rows are written.  (Refused before any CUDA work: runs without a GPU.)"""

import ctypes

import pytest

P = 1 << 30  # a fake aligned address, never read


@pytest.fixture(scope="module")
def M():
    from mixture_experts_layer_softmax_gb300 import _build
    _build.build()
    from mixture_experts_layer_softmax_gb300 import moe
    return moe


@pytest.mark.parametrize("T,h,K,dtype,size", [(16, 128, 2, 1, 2), (7, 1000, 1, 1, 2), (300, 36, 8, 0, 4)])
def test_rows_over_dy(M, T, h, K, dtype, size):
    f = M.raw("moe_unpermute_combine_bwd")
    r = ctypes.byref(M.make_config(T, h, 8, K, 8, dtype=dtype, flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_VALIDATE_ONLY))
    dy, rows = T * h * size, T * K * h * size
    up = lambda n: (n + 15) // 16 * 16  # noqa: E731
    for at in (P, P + 16, P + up(dy) - 16, P - 16, P - up(rows) + 16):
        assert f(r, P, None, P, None, at, None, None) == M.MOE_ERR_INVALID_ARG, at - P
    for at in (P + up(dy), P - up(rows), P + (1 << 28)):
        assert f(r, P, None, P, None, at, None, None) == M.MOE_OK, at - P


def test_without_tokens(M):
    f = M.raw("moe_unpermute_combine_bwd")
    r = ctypes.byref(M.make_config(0, 128, 8, 2, 8, flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_VALIDATE_ONLY))
    assert f(r, None, None, None, None, None, None, None) == M.MOE_OK
    assert f(r, P, None, P, None, P, None, None) == M.MOE_OK
