"""The write of a cache in 4 bits for units that are powers of two other than one, whose kernel does not divide:
every byte against the plain implementation."""
import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_ref import E4M3, place
from test_gpu_paged4 import run_append

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


def border_rows(dtype):
    """float64 [n, 16] blocks: quotients on and beside every border of two codes for scales of every significand,
    the largest element's sixth on and beside every border of two scales, zeros, the type's ends, infinities, NaN."""
    rng, rows = np.random.RandomState(5), []
    step = float(torch.finfo(dtype).eps)
    for byte in range(1, 127):
        s = E4M3[byte]
        ties = s * np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
        beside = np.concatenate([ties, ties * (1 + step), ties * (1 - step)])
        for _ in range(3):
            block = rng.choice(np.concatenate([beside, -beside, [0.0, -0.0]]), 16)
            block[rng.randint(16)] = 6 * s * rng.choice([-1, 1])
            rows.append(block)
        near = E4M3[byte:byte + 2].mean() if byte < 126 else s
        for x in (near * 6, near * 6 * (1 + step), near * 6 * (1 - step)):
            block = np.clip(rng.randn(16) * x / 4, -x, x)
            block[5] = x
            rows.append(block)
    rows += [rng.choice([0.0, -0.0], 16), rng.randn(16) * 1e-5, rng.randn(16) * 1e4]
    while len(rows) % 8:
        rows.append(rng.randn(16))
    return np.stack(rows)


def special_rows(dtype):
    rng, info = np.random.RandomState(6), torch.finfo(dtype)
    tiny, big, inf, nan = float(info.smallest_normal), float(info.max), np.inf, np.nan
    rows = []
    for special in ([0.0, -0.0], [tiny, -tiny, 0.0], [tiny / 8, -0.0], [tiny, 1.0], [big, -big, 1.0, tiny], [big / 4, -big / 64, 3.0],
                    [inf, 1.0, -3.0], [-inf, 5.0, big], [nan, 1.0, -2.0], [nan], [nan, inf, -inf], [1.0, 1e-3, -40.0]):
        block = rng.choice(special, 16)
        block[0] = special[0]
        rows += [block, block[::-1]]
    return np.stack(rows)


@pytest.mark.parametrize("dtype,k_unit,v_unit", [
    (BF, 0.5, 4.0), (BF, 2.0 ** -99, 2.0 ** 99), (BF, 2.0 ** -60, 2.0 ** 101), (BF, 2.0 ** -100, 2.0 ** 102), (BF, 2.0 ** 101, 1.0),
    (HF, 0.5, 4.0), (HF, 2.0 ** -6, 2.0 ** 4), (HF, 2.0 ** -99, 2.0 ** 99), (HF, 2.0 ** -60, 2.0 ** 101)])
def test_write_with_units_that_are_powers_of_two(dtype, k_unit, v_unit):
    blocks = border_rows(dtype)
    rows = [blocks, special_rows(dtype)]
    for unit in (k_unit, v_unit):  # quotients that the cache's codes resolve, where the type holds them
        with np.errstate(over="ignore"):
            rows.append(blocks * unit)
    x = np.concatenate(rows)
    x = x[:len(x) // 8 * 8].reshape(-1, 1, 128)
    k = torch.tensor(x, device="cuda").to(dtype)
    v = k.flip(0).contiguous()
    T = k.shape[0]
    codes, scales = place((T, 1, 1, 64), "tokens", 0x5a), place((T, 1, 1, 8), "tokens", 0x5a)
    run_append(k, v, torch.randperm(T, device="cuda"), codes, scales, 1, k_unit=k_unit, v_unit=v_unit)
