"""Workspace sizes over the number of tokens: one workspace, sized for the largest
batch, serves every smaller one through every call (no GPU needed)."""

import ctypes

import pytest

P = 1 << 20  # a fake aligned address, never read

CONFIGS = [
    dict(h=4096, E=8, K=2, F=14336),
    dict(h=7168, E=256, K=8, F=2048, n_shared=1),
    dict(h=2048, E=64, K=8, F=1024),
    dict(h=8, E=256, K=16, F=8),
]
TOKENS = (1, 2, 5, 8, 9, 31, 32, 33, 63, 64, 65, 66, 96, 128, 129, 176, 200, 256, 1000, 4096)


@pytest.fixture(scope="module")
def M():
    from mixture_experts_layer_softmax_gb300 import _build
    _build.build()
    from mixture_experts_layer_softmax_gb300 import moe
    return moe


def _cfg(M, **kw):
    return M.make_config(**dict(dict(flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_VALIDATE_ONLY), **kw))


def _calls(M, cfg, size):
    """The statuses of the calls that take a workspace, given `size` bytes of it."""
    r, sh = ctypes.byref(cfg), P if cfg.n_shared else None
    out = [M.raw("moe_layer_fwd")(r, P, P, None, None, P, None, P, None, sh, sh, P, None, None, P, size, None),
           M.raw("moe_router_topk")(r, P, P, None, None, None, P, P, None, P, size, None),
           M.raw("moe_permute")(r, P, P, P, P, P, P, P, P, P, P, size, None),
           M.raw("moe_grouped_mlp_fwd")(r, P, P, None, P, None, P, None, None, P, P, size, None)]
    if cfg.T <= 64:
        out.append(M.raw("moe_layer_fwd_few")(r, P, P, None, None, P, None, P, None, sh, sh, P, None,
                                              None, P, size, None))
        if cfg.h % 128 == 0 and cfg.F % 128 == 0:
            out.append(M.raw("moe_layer_fwd_few_mxfp4")(r, P, P, None, None, P, P, P, P, sh, sh, sh, sh, P,
                                                        None, None, P, size, None))
    return out


@pytest.mark.parametrize("kw", CONFIGS)
def test_sizes_do_not_shrink_as_tokens_are_added(M, kw):
    for extra in ({}, dict(flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_SAVE_FOR_BWD), dict(aux_loss_coeff=0.01),
                  dict(dtype=M.MOE_F32)):
        last = 0
        for T in TOKENS:
            n = M.moe_workspace_size(_cfg(M, T=T, **dict(kw, **extra)))
            assert n >= last and n % 256 == 0, (T, n, last)
            last = n


@pytest.mark.parametrize("kw", CONFIGS)
@pytest.mark.parametrize("most", [65, 128, 176])
def test_a_workspace_for_the_largest_batch_serves_smaller_ones(M, kw, most):
    size = M.moe_workspace_size(_cfg(M, T=most, **kw))
    for T in TOKENS:
        if T <= most:
            assert all(s == M.MOE_OK for s in _calls(M, _cfg(M, T=T, **kw), size)), T


def test_calls_without_a_few_token_form_need_only_their_own_bytes(M):
    """Batches past 64 tokens, and training configurations, which the few-token calls
    refuse: the bytes of the layer pass, as its buffers add up to them."""
    kw = dict(h=4096, E=8, K=2, F=14336)
    for T, size in ((65, 6_145_024), (128, 11_841_280)):
        assert all(s == M.MOE_OK for s in _calls(M, _cfg(M, T=T, **kw), size)), T
        assert M.raw("moe_layer_fwd")(ctypes.byref(_cfg(M, T=T, **kw)), P, P, None, None, P, None, P, None,
                                      None, None, P, None, None, P, size - 1, None) == M.MOE_ERR_WORKSPACE
    # 64 tokens more cost as much from 64 on as from 1024 on, to a few KB of rounding
    for extra in (dict(flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_SAVE_FOR_BWD), dict(z_loss_coeff=0.01)):
        n = {T: M.moe_workspace_size(_cfg(M, T=T, **dict(kw, **extra))) for T in (64, 128, 1024, 1088)}
        assert abs((n[128] - n[64]) - (n[1088] - n[1024])) < 65536
