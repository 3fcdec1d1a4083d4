"""The few-token calls' waits on counts run out: the call ends by itself, records the
timeout and writes no y, and the next call on the same workspace is right again."""

import pytest
import torch

from gpu_util import lib, needs_gpu
from test_gpu_few import Few

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("mx", [False, True])
def test_a_count_that_never_comes(mx, T, which):
    M = lib()
    f = Few(T=T, h=512, E=8, K=2, F=384, mx=mx, shared=1).device(M)
    torch.cuda.synchronize()
    assert M.moe_test_few_wait_runs_out(which) == 0
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_ERR_TIMEOUT
    assert M.moe_get_error() == M.MOE_OK
    assert torch.isnan(f.y).all()
    assert M.moe_test_few_wait_runs_out(0) == 0        # spent
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    f.check(M)
