"""moe_layer_fwd_few_mxfp4 with a second projection in several slices of F (more
than 4096 columns), whose stages hold 512 columns, and with long tokens."""

import pytest

from gpu_util import needs_gpu
from test_gpu_few_accuracy import Case, checked, only_the_output_rounding

pytestmark = [pytest.mark.gpu, needs_gpu]

CASES = [
    dict(T=3, h=256, E=2, K=1, F=4224),              # 33 blocks of 128: slices of 4 and 5 stages, the last of 128
    dict(T=20, h=256, E=2, K=2, F=4224, shared=1),   # units of 16 tokens
    dict(T=3, h=128, E=2, K=1, F=9088),              # 71 blocks: three slices, scale words not in fours
    dict(T=20, h=256, E=2, K=2, F=9088),
    dict(T=5, h=384, E=3, K=2, F=8704, shared=1),    # 68 blocks: scale words in fours
    dict(T=33, h=128, E=2, K=1, F=14336),            # four slices
    dict(T=2, h=7168, E=4, K=2, F=256),
    dict(T=17, h=7168, E=2, K=2, F=384),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"T{c['T']}_h{c['h']}_F{c['F']}")
def test_slices_and_long_tokens(c):
    f = checked(Case(mx=True, **c))
    if c["T"] * c["h"] >= 4096:
        only_the_output_rounding(f)
