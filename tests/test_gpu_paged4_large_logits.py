"""Attention over the cache in 4 bits with the largest logits that the contract allows (2^23 in log2 units): the
rounding of a row's maximum, half a step there, moves all of its weights alike and none out of fp16's range."""
import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_levels import Levels
from test_gpu_paged4 import run_fwd

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("gap", [3.0e5, 1.1 * 2.0 ** 22, 2.0 ** 24 / 2.1])
@pytest.mark.parametrize("q0", [1.0, -1.0])
@pytest.mark.parametrize("lens", [[(4000, 1)], [(300, 1)] * 160, [(1000, 5)] * 3, [(3500, 130)], [(300, 1)] * 20 + [(700, 200)]],
                         ids=["one", "many", "verify", "chunk", "mixed"])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (128, HF), (256, BF)])
def test_two_sizes_of_logits_far_apart(lens, D, dtype, q0, gap):
    """O is the value of the larger logits: all of them are one number, so their weights are equal and the others'
    are zero.  The larger logits are gap * ln 2, or -gap * ln 2 where every key has that."""
    for high in ((lambda j: j % 3 == 0), (lambda j: True)):
        b = Levels(lens, 2, 2, D, dtype, high, gap, 6.0, 2.0, q0=q0)
        o, lse = run_fwd(b)
        top = q0 > 0 or high(1)  # the larger logits are the high keys'
        want = 6.0 if top else 2.0625  # 2 in a cache: a sixth of it is nearest to a scale of 0.34375, times 6
        assert torch.equal(o, torch.full_like(o, want))
        z = q0 * 6 * b.scale if top else 0.0
        # the logit and the product with ln 2 are rounded, once each, and the sum of n weights is off by n / 2^24
        n = np.array([sum(high(j) == top for j in range(kv - x + t + 1)) for kv, x in lens for t in range(x)])
        exact = z + np.log(n)
        assert (np.abs(lse.double().cpu().numpy() - exact) <= 2.0 ** -21 * (1 + np.abs(exact)) + n * 2.0 ** -23).all()
