"""attn_paged_free on block tables around and above the size from which two kernels do its work."""
import random

import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_ref import random_rows
from test_gpu_pages import dev, ok, run_free

pytestmark = pytest.mark.gpu
I32 = torch.int32
LARGE = 65536  # entries


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


@pytest.mark.parametrize("n,width,page,hi", [(64, 1023, 16, 900), (64, 1024, 16, 900), (1, LARGE - 1, 1, 60000), (1, 70000, 1, 70000),
                                             (LARGE, 1, 4, 4), (300, 400, 7, 500), (2500, 40, 16, 600), (1100, 70, 64, 4400)])
@pytest.mark.parametrize("shared", [False, True])
def test_free_of_wide_and_tall_tables(n, width, page, hi, shared):
    rng = random.Random(n + width)
    n_pages = n * (hi // page + 1) + 50
    kv, table, rest = random_rows(rng, n, page, hi, width, n_pages)
    shares = [0] * n_pages
    if shared:
        for i in range(n):
            j = rng.randrange(n)
            m = rng.randint(0, min(kv[i], kv[j]) // page)
            table[i][:m] = table[j][:m]
        for row, x in zip(table, kv):
            for col in range(-(-x // page)):
                shares[row[col]] += 1
        shares = [max(x - 1, 0) + (rng.random() < 0.05) for x in shares]
    for keep in ([0] * n, [max(0, x - rng.randint(0, 20)) for x in kv], [rng.randint(-5, hi + 5) for _ in kv], kv):
        taken = n_pages - len(rest)
        run_free(kv, keep, table, page, shares, [-5] * taken + rest, taken, stride=rng.choice([None, width + 2]))


def test_free_of_a_wide_table_is_the_same_in_every_run():
    """More names than counts, on the default stream, on another, and in a replayed graph."""
    n, page = 600, 16
    table = torch.randint(0, 9000, (n, 120), dtype=I32, device="cuda")
    assert table.numel() >= LARGE
    kv, keep, head = torch.full((n,), 1920, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda"), dev([9000])
    shares, free = torch.empty(9000, dtype=I32, device="cuda"), torch.empty(9000, dtype=I32, device="cuda")
    counts, outs = torch.empty(4, dtype=I32, device="cuda"), []

    def fresh():
        shares.fill_(7)
        free.zero_()
        counts.zero_()
        torch.cuda.synchronize()

    def done():
        torch.cuda.synchronize()
        ok()
        outs.append((shares.tolist(), free.tolist(), counts.tolist()))

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for stream in (None, side, None, side):
        fresh()
        fa.attn_paged_free(kv, keep, table, page, shares, free, head, counts=counts, stream=stream)
        done()
    with torch.cuda.graph(graph):
        fa.attn_paged_free(kv, keep, table, page, shares, free, head, counts=counts)
    for _ in range(3):
        fresh()
        graph.replay()
        done()
    names = torch.bincount(table.flatten().long(), minlength=9000)
    freed = (names > 7).nonzero().flatten().tolist()
    assert 0 < len(freed) < 9000
    left = torch.where(names > 7, 0, 7 - names).tolist()
    assert all(x == (left, [0] * (9000 - len(freed)) + freed, [len(freed), 9000 - len(freed), 0, 0]) for x in outs)


def test_free_takes_the_kernels_that_the_header_names():
    kv, keep, counts = dev([5]), dev([0]), dev([0] * 4)
    for width, kernels in ((LARGE - 1, 1), (LARGE, 2)):
        table = torch.zeros((1, width), dtype=I32, device="cuda")
        before = fa.attn_kernel_launches()
        fa.attn_paged_free(kv, keep, table, 16, dev([0]), dev([-1]), dev([1]), counts=counts)
        ok()
        assert fa.attn_kernel_launches() - before == kernels and counts.tolist() == [1, 0, 0, 0]
