"""Attention over the cache in 4 bits whose bf16 query rows are zero or nearly so, at small and large
softmax scales: every logit is (nearly) zero and O is the mean of the seen values."""
import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
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


SCALES = [(2.0 ** -24, 1.0), (2.0 ** -30, 1.0), (0.088, 1e-7), (2.0 ** -120, 1.0)]


@pytest.mark.parametrize("D,dtype,scale,k_unit", [(D, t, *s) for D, t in ((64, BF), (128, BF), (256, BF), (128, HF)) for s in SCALES] +
                         [(D, BF, 2.0 ** 60, 1.0) for D in (64, 128, 256)])  # with fp16's numbers past the largest logits
@pytest.mark.parametrize("lens", [DECODE, VERIFY, MIXED], ids=["decode", "verify", "mixed"])
def test_rows_of_zeros_and_of_tiny_numbers(lens, D, dtype, scale, k_unit):
    b = Batch4(lens, 4, 2, D, 16, dtype, k_unit=k_unit, pad_rows=1, seed=D)
    b.scale = scale
    # of every four rows one of zeros, one of the smallest normal sizes, one with a single tiny element
    kind = torch.arange(b.q.shape[0] * 4).reshape(-1, 4, 1) % 4
    tiny = 2.0 ** -120 if dtype is BF else 2.0 ** -24
    one = torch.where(torch.arange(D) == D // 3, tiny, 0.0).expand_as(b.q)
    rest = b.q.float() * (2.0 ** -70 if scale > 1 else 1.0)
    b.q = torch.where(kind == 0, 0.0, torch.where(kind == 1, tiny * b.q.float().sign(), torch.where(kind == 2, one, rest))).to(dtype)
    check(b, *run_fwd(b), untouched=9.0)


@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
def test_keys_of_zeros_under_large_queries(lens):
    """Logits of zero whose row's scale is past fp32's range."""
    b = Batch4(lens, 4, 2, 128, 16, seed=1)
    b.q, b.scale = b.q * 2.0 ** 100, 2.0 ** 60
    b.k_scales.fill_(0)
    b.dense = [(np.zeros_like(k), v) for k, v in b.dense]
    check(b, *run_fwd(b))
