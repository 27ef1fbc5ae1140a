"""CPU-only: the softmax scale of attention over the cache in 4 bits has to be a normal number of fp32."""
import pytest

import attention_forward_11_gb300 as fa
from attention_forward_11_gb300 import build as fa_build
from test_paged4_host import FWD, ids


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    fa.load_library()


@pytest.mark.parametrize("over", [dict(scale=1e-20, ku=1e-20), dict(scale=8e-39), dict(scale=0.088, ku=8e-38), dict(scale=1e-43)], ids=ids)
def test_scales_that_fp32_holds_with_few_bits_are_refused(over):
    assert fa.attn_paged_coded_fwd_ptr(*{**FWD, **over}.values()) == fa.ATTN_ERR_INVALID_ARG
