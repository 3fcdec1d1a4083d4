"""A tensor of another element type than the call reads or writes is refused by the
binding, before its address is taken: a bf16 norm weight, say, would be read as fp32 past
its end.  (Addresses given as integers have no type; a refusal comes before any CUDA call,
so these run without a GPU.)"""

import pytest
import torch

P = 1 << 20  # a fake aligned address, never read

CALLS = {  # the call, its leading arguments, and each tensor's type: b(ytes of codes), f(p32), h(bf16), i(nt32)
    "moe_fp8_quantize": ((4, 128), "hbf"),
    "moe_fp8_quantize_weights": ((1, 128, 128), "hbfbf"),
    "moe_permute_fp8": ("cfg", "bfifbfiiiif"),
    "moe_expert_fc1_fp8": ("cfg", "bfifbfhhbf"),
    "moe_expert_fc2_fp8": ("cfg", "bfibfh"),
    "moe_rmsnorm_fwd": ((4, 128, 1), "hhf-hhbff"),
    "moe_rmsnorm_bwd": ((4, 128, 1), "hhffhhf"),
    "moe_unpermute_combine_bwd": ("cfg", "hhifhf"),
}
TYPES = {"b": torch.uint8, "f": torch.float32, "h": torch.bfloat16, "i": torch.int32}
ALL = (torch.uint8, torch.float32, torch.bfloat16, torch.int32, torch.float16, torch.int64, torch.float64)


@pytest.fixture(scope="module")
def M():
    from mixture_experts_layer_softmax_gb300 import _build
    _build.build()
    from mixture_experts_layer_softmax_gb300 import moe
    return moe


def _args(M, name, k, tensor):
    head, kinds = CALLS[name]
    head = [M.make_config(4, 128, 4, 2, 128)] if head == "cfg" else list(head)
    args = [P if kind != "-" else 1e-6 for kind in kinds]
    args[k] = tensor
    return head + args + ([None] if name == "moe_permute_fp8" else [])   # its workspace


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_of_every_call(M, name):
    kinds = CALLS[name][1]
    for k, kind in enumerate(kinds):
        if kind == "-":
            continue
        for dtype in ALL:
            if dtype == TYPES[kind]:
                continue
            with pytest.raises(ValueError, match="expected .* not torch"):
                getattr(M, name)(*_args(M, name, k, torch.zeros(4, 128, dtype=dtype)))
        # of its own type the refusal is about where it lies
        with pytest.raises(ValueError, match="CUDA tensor"):
            getattr(M, name)(*_args(M, name, k, torch.zeros(4, 128, dtype=TYPES[kind])))


def test_codes_may_have_the_formats_own_type(M):
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.moe_fp8_quantize(4, 128, P, torch.zeros(4, 128).to(torch.float8_e4m3fn), P)


def test_fp32_calls_take_fp32_rows(M):
    for k in (0, 1, 4, 5):
        args = [P, P, P, 1e-6, P, P]
        args[k] = torch.zeros(4, 128, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="expected .* not torch.bfloat16"):
            M.moe_rmsnorm_fwd(4, 128, M.MOE_F32, *args)
    cfg = M.make_config(4, 128, 4, 2, 128, dtype=M.MOE_F32)
    with pytest.raises(ValueError, match="expected .* not torch.bfloat16"):
        M.moe_unpermute_combine_bwd(cfg, torch.zeros(4, 128, dtype=torch.bfloat16), None, P, None, P)
