"""Attention over the cache in 4 bits with units of V near the ends of fp32's range: O is representable, sums of
weighted values times the unit, or the unit over a row's sum, need not be."""
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_levels import Levels
from paged_ref import check
from test_gpu_paged4 import run_fwd

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("lens", [[(20000, 1)], [(20000, 1)] * 3, [(1500, 1)] * 160, [(6000, 5)] * 3, [(17000, 64)],
                                  [(900, 260)] * 4, [(1500, 1)] * 20 + [(900, 300)]],
                         ids=["one", "three", "many", "verify", "chunk", "prompts", "mixed"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("exponent", [124, -120])
def test_units_near_the_ends(lens, D, exponent):
    """O is in bf16's range; sums of weighted values times the unit need not be."""
    b = Levels(lens, 2, 2, D, BF, lambda j: j % 3 == 0, 3.0, 2.0, 6.0, v_unit=2.0 ** exponent)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("lens", [[(20000, 1)], [(1500, 1)] * 160, [(9000, 64)], [(900, 260)] * 4], ids=["one", "many", "chunk", "prompts"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_units_under_large_sums(lens, D):
    """Logits that rise after a row's first keys, by less than what rescales its sums; O is a normal number, the
    unit over a row's sum is none."""
    b = Levels(lens, 2, 2, D, BF, lambda j: j >= 200, 14.0, 448.0, 6.0, v_unit=2.0 ** -127)
    check(b, *run_fwd(b))
