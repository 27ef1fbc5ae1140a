"""GPU parity of the forward on logits far from zero: the weights of a row are relative to
its own maximum, however far below zero that is (fp16 weights relative to zero would
vanish below 2^-24)."""
import math

import numpy as np
import pytest

from attention_forward_11_gb300 import inputs
from parity import compare, run_gpu
import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [-60.0, -17.3, 40.0])
@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "f16"), (256, "f16"), (64, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 2, 1, 1), (300, 300, 4, 2), (130, 700, 2, 2)])
def test_logits_far_from_zero(shape, D, dtype, shift):
    Sq, Skv, Hq, Hkv = shape
    q, k, v = inputs.make_qkv(1, Sq, Skv, Hq, Hkv, D, seed=D + Sq, dtype=dtype)
    scale = 1 / math.sqrt(D)
    values = np.array([16.0, shift * math.sqrt(D) / 16], dtype=np.float32)  # every logit is moved by about `shift`
    bits = values.astype(np.float16).view(np.uint16) if dtype == "f16" else inputs.f32_to_bf16_bits(values)
    q[..., 0], k[..., 0] = bits
    o, lse = run_gpu(q, k, v, 1, scale, dtype=dtype)
    ro, rl = oracle.attn_full(q, k, v, 1, scale, f16=dtype == "f16")
    compare(o, lse, ro, rl, str((shape, D, dtype, shift)), dtype)
