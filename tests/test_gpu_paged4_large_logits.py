"""Attention over the cache in 4 bits with logits so large that a step of fp32 between them is a factor of a weight:
weights are relative to the row's own maximum and never past it."""
import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_levels import Levels
from paged4_ref import Batch4
from paged_ref import check
from test_gpu_paged4 import DECODE, MIXED, VERIFY, run_fwd

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("gap", [3.0e5, 1.1 * 2.0 ** 22, 7.3 * 2.0 ** 25, 2.0 ** 30 / 3, 1.7 * 2.0 ** 45, 1.2 * 2.0 ** 100])
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


@pytest.mark.parametrize("scale", [2.0 ** 24, 2.0 ** 60])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (256, BF), (128, HF)])
@pytest.mark.parametrize("lens", [DECODE, VERIFY, MIXED], ids=["decode", "verify", "mixed"])
def test_logits_of_many_sizes(lens, D, dtype, scale):
    """Rows from fp16's smallest numbers on: O stays among the values of the keys that are seen."""
    b = Batch4(lens, 4, 2, D, 16, dtype, pad_rows=1, seed=D)
    b.scale = scale
    b.q = (b.q.float() * 2.0 ** (-24 + 8.0 * (torch.arange(b.q.shape[0] * 4) % 4).reshape(-1, 4, 1))).to(dtype)
    o, lse = run_fwd(b)
    check(b, o, lse, untouched=9.0)
    at = 0
    for (kv, n), (_, v) in zip(lens, b.dense):
        for t in range(n):
            seen = np.repeat(np.asarray(v)[:kv - n + t + 1], 2, axis=1)
            x = o[at + t].double().cpu().numpy()
            step = 2.0 ** -7 * np.abs(seen).max(axis=0)
            assert (x <= seen.max(axis=0) + step).all() and (x >= seen.min(axis=0) - step).all()
        at += n
