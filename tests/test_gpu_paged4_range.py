"""Attention over the cache in 4 bits where weights take a wide range of sizes: many keys far below a few (a
prompt's first token, say)."""
import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_levels import Levels
from paged_ref import U
from test_gpu_paged4 import run_fwd

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("lens", [[(4000, 1)], [(1500, 1)] * 80, [(2900, 5)] * 3, [(3500, 260)], [(1500, 1)] * 30 + [(900, 300)]],
                         ids=["one", "many", "verify", "chunk", "mixed"])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (128, HF), (256, BF)])
def test_many_keys_far_below_a_few(lens, D, dtype):
    """Weights of 2^-25.5 of the largest, but for every 224th: together they are all of O, since the values at the
    largest are zero.  The bound is paged4_ref.py's (with A = sum P |v| = O) but for the weights that lie below
    fp16's normal numbers: relative to a maximum of at least 2^7 they are held to half of 2^-24, 2^-32 of it."""
    b = Levels(lens, 4, 2, D, dtype, lambda j: j % 224 == 3, 25.5, 0.0, 448.0)
    o, lse = run_fwd(b)
    ro, rl, _, tol_l = b.reference()
    o = o.double().cpu().numpy()
    e = 4 * D * 2.0 ** -24 * b.scale * 6
    at = 0
    for kv, n in lens:
        for t in range(n):
            seen = kv - n + t + 1
            few = -(-(seen - 3) // 224)
            want = ro[at + t]
            tol = (2.0 ** -11 + 2 * e + 2 * kv * 2.0 ** -24 + 2.0 ** -19 + U[dtype]) * want + 2.0 ** -32 * 448 * seen / few
            assert (np.abs(o[at + t] - want) <= tol).all(), (at + t, o[at + t].max(), want.max(), tol.max())
        at += n
    assert (np.abs(lse.double().cpu().numpy() - rl) <= tol_l).all()
