"""Argument checks of the MXFP4 calls and of the layer for a few tokens: every
refusal comes before any CUDA call, so these run without a GPU."""

import ctypes

import pytest

P = 1 << 20  # a fake aligned address, never read


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


def test_quantize_and_dequantize(M):
    for name in ("moe_mxfp4_quantize", "moe_mxfp4_dequantize"):
        f = M.raw(name)
        assert f(10, 96, 1, None, P, P, P, None) == M.MOE_ERR_UNSUPPORTED
        assert f(10, 0, 1, None, P, P, P, None) == M.MOE_ERR_INVALID_ARG
        assert f(-1, 128, 1, None, P, P, P, None) == M.MOE_ERR_INVALID_ARG
        assert f(1 << 32, 128, 1, None, P, P, P, None) == M.MOE_ERR_INVALID_ARG
        assert f(10, 128, 3, None, P, P, P, None) == M.MOE_ERR_INVALID_ARG   # 10 % 3 != 0
        assert f(10, 128, 0, None, P, P, P, None) == M.MOE_ERR_INVALID_ARG
        assert f(10, 128, 300, P, P, P, P, None) == M.MOE_ERR_INVALID_ARG    # > 256 groups
        for k in range(3):
            for bad in (None, P + 8):
                a = [P, P, P]
                a[k] = bad
                assert f(10, 128, 1, None, *a, None) == M.MOE_ERR_INVALID_ARG
        assert f(0, 128, 1, None, None, None, None, None) == M.MOE_OK


def test_products(M):
    f1, f2 = M.raw("moe_expert_fc1_mxfp4"), M.raw("moe_expert_fc2_mxfp4")
    ok = _cfg(M)
    r = ctypes.byref(ok)
    assert f1(r, P, P, P, None, P, P, P, None, None, None) == M.MOE_OK
    assert f1(r, P, P, P, None, P, P, None, P, P, None) == M.MOE_OK
    assert f1(r, P, P, P, None, P, P, None, None, None, None) == M.MOE_ERR_INVALID_ARG  # no output
    assert f1(r, P, P, P, None, P, P, None, P, None, None) == M.MOE_ERR_INVALID_ARG
    assert f1(r, P, P, None, None, P, P, P, None, None, None) == M.MOE_ERR_INVALID_ARG
    assert f1(r, P + 4, P, P, None, P, P, P, None, None, None) == M.MOE_ERR_INVALID_ARG
    assert f2(r, P, P, P, P, P, P, None) == M.MOE_OK
    assert f2(r, P, None, P, P, P, P, None) == M.MOE_ERR_INVALID_ARG
    assert f2(r, P, P, P, P, P, P + 2, None) == M.MOE_ERR_INVALID_ARG
    for kw in (dict(act=M.MOE_ACT_GELU), dict(F=192), dict(h=200), dict(dtype=M.MOE_F32)):
        bad = ctypes.byref(_cfg(M, **kw))
        assert f1(bad, P, P, P, None, P, P, P, None, None, None) == M.MOE_ERR_UNSUPPORTED
        assert f2(bad, P, P, P, P, P, P, None) == M.MOE_ERR_UNSUPPORTED


def _few(M, cfg, ws=P, size=1 << 40, **kw):
    a = dict(x=P, w_r=P, gb=None, sb=None, w1=P, b1=None, w2=P, b2=None, w1s=None, w2s=None, y=P,
             idx=None, prob=None)
    a.update(kw)
    return M.raw("moe_layer_fwd_few")(ctypes.byref(cfg), *a.values(), ws, size, None)


def _few4(M, cfg, ws=P, size=1 << 40, **kw):
    a = dict(x=P, w_r=P, gb=None, sb=None, w1=P, w1f=P, w2=P, w2f=P, w1s=None, w1sf=None, w2s=None,
             w2sf=None, y=P, idx=None, prob=None)
    a.update(kw)
    return M.raw("moe_layer_fwd_few_mxfp4")(ctypes.byref(cfg), *a.values(), ws, size, None)


@pytest.mark.parametrize("call", [_few, _few4])
def test_few_tokens(M, call):
    assert call(M, _cfg(M)) == M.MOE_OK
    assert call(M, _cfg(M, T=64)) == M.MOE_OK
    assert call(M, _cfg(M, T=0), x=None, y=None) == M.MOE_OK
    assert call(M, _cfg(M, capacity=3, flags=M.MOE_FLAG_VALIDATE_ONLY)) == M.MOE_OK
    for kw in (dict(T=65), dict(dtype=M.MOE_F32), dict(aux_loss_coeff=0.1), dict(z_loss_coeff=0.1),
               dict(flags=M.MOE_FLAG_SAVE_FOR_BWD | M.MOE_FLAG_VALIDATE_ONLY), dict(E=300)):
        assert call(M, _cfg(M, **kw)) == M.MOE_ERR_UNSUPPORTED
    huge = _cfg(M, T=64, K=8, h=1 << 20, F=1 << 20)                # units past 31 bits
    assert call(M, huge) == M.MOE_ERR_UNSUPPORTED
    for kw in (dict(K=9), dict(T=-1), dict(capacity=-1)):
        assert call(M, _cfg(M, **kw)) == M.MOE_ERR_INVALID_ARG
    for name in ("x", "w_r", "w1", "w2", "y"):
        assert call(M, _cfg(M), **{name: None}) == M.MOE_ERR_INVALID_ARG
        assert call(M, _cfg(M), **{name: P + 8}) == M.MOE_ERR_INVALID_ARG
    need = M.moe_workspace_size(_cfg(M))
    assert call(M, _cfg(M), size=need) == M.MOE_OK
    assert call(M, _cfg(M), size=need - 1) == M.MOE_ERR_WORKSPACE
    assert call(M, _cfg(M), ws=None) == M.MOE_ERR_WORKSPACE
    assert call(M, _cfg(M), ws=P + 128) == M.MOE_ERR_INVALID_ARG
    shared = _cfg(M, n_shared=1)
    assert call(M, shared) == M.MOE_ERR_INVALID_ARG


def test_few_tokens_weights(M):
    biased = _cfg(M, act=M.MOE_ACT_GELU, has_bias=1)
    assert _few(M, biased) == M.MOE_ERR_INVALID_ARG
    assert _few(M, biased, b1=P, b2=P) == M.MOE_OK
    assert _few(M, _cfg(M, n_shared=1), w1s=P, w2s=P) == M.MOE_OK
    assert _few(M, _cfg(M, h=136, F=72)) == M.MOE_OK
    for kw in (dict(h=136), dict(F=72), dict(act=M.MOE_ACT_GELU)):
        assert _few4(M, _cfg(M, **kw)) == M.MOE_ERR_UNSUPPORTED
    for name in ("w1f", "w2f"):
        assert _few4(M, _cfg(M), **{name: None}) == M.MOE_ERR_INVALID_ARG
        assert _few4(M, _cfg(M), **{name: P + 4}) == M.MOE_ERR_INVALID_ARG
    sh = dict(w1s=P, w1sf=P, w2s=P, w2sf=P)
    assert _few4(M, _cfg(M, n_shared=1), **sh) == M.MOE_OK
    assert _few4(M, _cfg(M, n_shared=1), **dict(sh, w2sf=None)) == M.MOE_ERR_INVALID_ARG


def test_workspace_covers_both_calls(M):
    """The few-token scratch fits the workspace of every config it accepts, and
    the size does not shrink as tokens are added."""
    for kw in (dict(h=7168, E=256, K=8, F=2048), dict(h=4096, E=8, K=2, F=14336),
               dict(h=8, E=256, K=16, F=8), dict(h=2048, E=64, K=8, F=1024, n_shared=1)):
        last = 0
        for T in (1, 2, 7, 8, 9, 16, 17, 32, 33, 64):
            n = M.moe_workspace_size(_cfg(M, T=T, **kw))
            assert n >= last and n % 256 == 0
            last = n


def test_wait_hook(M):
    """What is pending is handed back, and calls that enqueue nothing leave it."""
    assert M.moe_test_few_wait_runs_out(3) == -1 and M.moe_test_few_wait_runs_out(-1) == -1
    assert M.moe_test_few_wait_runs_out(2) == 0
    assert _few(M, _cfg(M)) == M.MOE_OK                            # validates only
    assert _few(M, _cfg(M, T=0, flags=0), x=None, y=None) == M.MOE_OK
    assert M.moe_test_few_wait_runs_out(1) == 2
    assert M.moe_test_few_wait_runs_out(0) == 1
    assert M.moe_test_few_wait_runs_out(0) == 0
