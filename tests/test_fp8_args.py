"""Argument checks of the FP8 layer path's calls: every refusal comes before any
CUDA call, so these run without a GPU."""

import ctypes

import pytest

P = 1 << 20  # a fake aligned address, never read
BIG = 1 << 40


@pytest.fixture(scope="module")
def M():
    from mixture_experts_layer_softmax_gb300 import _build
    _build.build()
    from mixture_experts_layer_softmax_gb300 import moe
    return moe


def _cfg(M, **kw):
    base = dict(T=16, h=128, E=8, K=2, F=256, flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_VALIDATE_ONLY)
    base.update(kw)
    return M.make_config(**base)


def _each_bad(good, which, values):
    for k in which:
        for bad in values:
            a = list(good)
            a[k] = bad
            yield a


def test_quantizers(M):
    f = M.raw("moe_fp8_quantize")
    assert f(10, 96, P, P, P, None) == M.MOE_ERR_UNSUPPORTED
    assert f(10, 0, P, P, P, None) == M.MOE_ERR_INVALID_ARG
    assert f(-1, 128, P, P, P, None) == M.MOE_ERR_INVALID_ARG
    assert f(1 << 32, 128, P, P, P, None) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad([P, P, P], range(3), (None, P + 8)):
        assert f(10, 128, *a, None) == M.MOE_ERR_INVALID_ARG
    assert f(0, 128, None, None, None, None) == M.MOE_OK
    g = M.raw("moe_fp8_quantize_weights")
    for G, N, K, st in ((0, 128, 128, 1), (1, 0, 128, 1), (1, 128, -128, 1), (1, 64, 128, 2), (1, 128, 200, 2),
                        (1 << 20, 1 << 20, 128, 2), (2, 1 << 30, 1 << 30, 2)):
        assert g(G, N, K, P, P, P, P, P, None) == st, (G, N, K)
    for a in _each_bad([P, P, P, P, P], range(5), (P + 4,)):
        assert g(1, 128, 128, *a, None) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad([P, P, P, P, P], range(5), (None,)):   # q_t and sf_t: both or neither
        assert g(1, 128, 128, *a, None) == M.MOE_ERR_INVALID_ARG


def test_permute(M):
    f = M.raw("moe_permute_fp8")
    ok = _cfg(M)
    good = [P] * 10 + [None]
    assert f(ctypes.byref(ok), *good, P, BIG, None) == M.MOE_OK            # no perm_prob
    for a in _each_bad(good, (0, 1, 2, 4, 5, 6, 7, 8, 9), (None,)):
        assert f(ctypes.byref(ok), *a, P, BIG, None) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad(good, (0, 1, 4, 5), (P + 8,)):
        assert f(ctypes.byref(ok), *a, P, BIG, None) == M.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(ok), *good, None, 0, None) == M.MOE_ERR_WORKSPACE
    assert f(None, *good, P, BIG, None) == M.MOE_ERR_INVALID_ARG
    for kw in (dict(h=200), dict(dtype=M.MOE_F32)):
        assert f(ctypes.byref(_cfg(M, **kw)), *good, P, BIG, None) == M.MOE_ERR_UNSUPPORTED


def test_products(M):
    f1, f2 = M.raw("moe_expert_fc1_fp8"), M.raw("moe_expert_fc2_fp8")
    r = ctypes.byref(_cfg(M))
    for tail, st in (((P, P, P, P), 0), ((None, P, None, None), 0), ((None, None, P, P), 0), ((P, None, None, None), 1),
                     ((None, P, P, None), 1), ((None, P, None, P), 1), ((P + 8, P, None, None), 1)):
        assert f1(r, P, P, P, None, P, P, *tail, None) == st, tail
    for a in _each_bad([P, P, P, P, P, P], (0, 1, 2, 4, 5), (None,)):
        assert f1(r, *a, None, P, None, None, None) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad([P, P, P, P, P, P], (0, 1, 4, 5), (P + 4,)):
        assert f1(r, *a, None, P, None, None, None) == M.MOE_ERR_INVALID_ARG
    assert f2(r, P, P, P, P, P, P, None) == M.MOE_OK
    for a in _each_bad([P] * 6, range(6), (None,)):
        assert f2(r, *a, None) == M.MOE_ERR_INVALID_ARG
    for kw in (dict(act=M.MOE_ACT_GELU), dict(F=192), dict(h=200), dict(dtype=M.MOE_F32)):
        bad = ctypes.byref(_cfg(M, **kw))
        assert f1(bad, P, P, P, None, P, P, None, P, None, None, None) == M.MOE_ERR_UNSUPPORTED
        assert f2(bad, P, P, P, P, P, P, None) == M.MOE_ERR_UNSUPPORTED


def test_rmsnorm(M):
    f, b = M.raw("moe_rmsnorm_fwd"), M.raw("moe_rmsnorm_bwd")
    fwd = lambda rows=4, h=256, dt=1, a=(P, P, P), eps=1e-6, o=(P, P, P, P, P): f(rows, h, dt, *a, eps, *o, None)  # noqa: E731
    assert fwd(rows=0, a=(None,) * 3, o=(None,) * 5) == M.MOE_OK
    for kw, st in ((dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(h=0), 1), (dict(dt=2), 1), (dict(h=12), 2),
                   (dict(h=6, dt=0), 2), (dict(h=65544), 2), (dict(h=200), 2), (dict(eps=-1e-6), 1),
                   (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(a=(None, P, P)), 1),
                   (dict(a=(P, P, None)), 1), (dict(o=(P, None, None, None, P)), 1), (dict(o=(P, P, P, None, P)), 1),
                   (dict(o=(P, P, None, P, P)), 1)):
        assert fwd(**kw) == st, kw
    for k in range(3):
        assert fwd(a=tuple(P + 8 if i == k else P for i in range(3))) == M.MOE_ERR_INVALID_ARG
    for k in range(5):
        assert fwd(o=tuple(P + 8 if i == k else P for i in range(5))) == M.MOE_ERR_INVALID_ARG
    size = M.moe_rmsnorm_bwd_workspace_size
    assert size(10, 256) >= 10 * 256 * 4 and size(10, 256) % 256 == 0
    assert size(0, 256) == 0 and size(-1, 256) == 0 and size(10, 6) == 0
    assert all(size(n, 4096) <= size(n + 1, 4096) for n in range(600)) and size(1 << 30, 4096) == size(1 << 20, 4096)
    need = size(4, 256)
    bwd = lambda rows=4, h=256, dt=1, a=(P, P, P, P, P, P, P), ws=P, n=need: b(rows, h, dt, *a, ws, n, None)  # noqa: E731
    for kw, st in ((dict(rows=-1), 1), (dict(h=0), 1), (dict(dt=5), 1), (dict(h=12), 2), (dict(ws=None), 3),
                   (dict(n=need - 1), 3), (dict(ws=P + 128), 1)):
        assert bwd(**kw) == st, kw
    for a in _each_bad([P] * 7, (0, 1, 2, 3, 5), (None, P + 8)):
        assert bwd(a=tuple(a)) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad([P] * 7, (4, 6), (P + 8,)):
        assert bwd(a=tuple(a)) == M.MOE_ERR_INVALID_ARG
    assert bwd(rows=0, a=(None,) * 7, ws=None, n=0) == M.MOE_OK


def test_combine_bwd(M):
    f = M.raw("moe_unpermute_combine_bwd")
    Q = P + 4096
    r = ctypes.byref(_cfg(M))
    assert f(r, P, P, P, None, Q, P, None) == M.MOE_OK
    assert f(r, P, None, P, P, Q, None, None) == M.MOE_OK
    assert f(r, P, P, P, P, Q, None, None) == M.MOE_ERR_INVALID_ARG       # y_perm without dprob
    assert f(r, P, None, P, P, Q, P, None) == M.MOE_ERR_INVALID_ARG
    assert f(r, P, Q, P, P, Q, P, None) == M.MOE_ERR_INVALID_ARG          # one buffer for both
    for a in _each_bad([P, P, P, P, Q, P], (0, 2, 4), (None,)):
        assert f(r, *a, None) == M.MOE_ERR_INVALID_ARG
    for a in _each_bad([P, P, P, P, Q, P], (0, 1, 4), (P + 8,)):
        assert f(r, *a, None) == M.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [
    lambda M: M.raw("moe_fp8_quantize")(10, 128, P, P, P, None),
    lambda M: M.raw("moe_fp8_quantize_weights")(1, 128, 128, P, P, P, None, None, None),
    lambda M: M.raw("moe_rmsnorm_fwd")(4, 256, 1, P, None, P, 1e-6, None, P, None, None, None, None),
    lambda M: M.raw("moe_rmsnorm_bwd")(4, 256, 1, P, P, P, P, None, P, None, None, 0, None),
    lambda M: M.raw("moe_unpermute_combine_bwd")(ctypes.byref(_cfg(M, flags=0)), P, None, P, P, P, None, None),
    lambda M: M.raw("moe_expert_fc2_fp8")(ctypes.byref(_cfg(M, flags=0)), P, P, P, P, P, P, None),
])
def test_injected_failure_comes_before_any_work(M, call):
    M.moe_test_inject_cuda_failure(1)
    assert call(M) == M.MOE_ERR_CUDA
    assert M.moe_test_inject_cuda_failure(0) == 0
