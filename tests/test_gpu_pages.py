"""Forking, freeing and copying the pages of a paged cache on the GPU, against their definitions."""
import random

import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_ref import plain_fork, plain_free, random_rows

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


def ok():
    assert fa.attn_check_device_status() == fa.ATTN_OK


def dev(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def wide_table(table, stride):
    t = torch.full((len(table), stride or len(table[0])), 77, dtype=I32, device="cuda")
    t[:, :len(table[0])] = dev(table)
    return t, t[:, :len(table[0])]


# ------------------------------------------------------------------ fork
def run_fork(parents, lens, kv, free, head, table, page, shares, stride=None, **kw):
    room, t = wide_table(table, stride)
    k, s = dev(kv), dev(shares)
    copies, counts = fa.attn_paged_fork(dev(parents), k, dev(free), t, page, s, lens=None if lens is None else dev(lens),
                                        free_head=None if head is None else dev([head]), **kw)
    ok()
    want = plain_fork(parents, lens, kv, free, head or 0, table, page, shares)
    for name, a, b in zip(("kv", "table", "shares", "copies", "counts"), (k, t, s, copies, counts), want):
        assert a.tolist() == b, name
    if stride:
        assert (room[:, len(table[0]):] == 77).all()
    return want


@pytest.mark.parametrize("n,page,hi", [(1, 16, 100), (2, 1, 9), (3, 16, 100), (40, 7, 300), (64, 16, 900), (257, 64, 2000),
                                       (1024, 16, 300), (1025, 32, 200), (2500, 16, 60)])
@pytest.mark.parametrize("part", [False, True])
def test_fork(n, page, hi, part):
    rng = random.Random(n + page)
    width = hi // page + 3
    kv, table, rest = random_rows(rng, n, page, hi, width, n * (hi // page + 1) + 60)
    # some rows go on from others, a few of them from rows that are forks themselves
    parents = [rng.choice([-1, i, rng.randrange(n), rng.randrange(max(1, n // 2))]) for i in range(n)]
    lens = [rng.choice([rng.randint(-3, hi + 10), 0, page, 2 * page]) for _ in range(n)] if part else None
    shares = [rng.choice([0, 0, 2]) for _ in range(n * (hi // page + 1) + 60)]
    run_fork(parents, lens, kv, rest, rng.choice([None, 2]), table, page, shares, stride=rng.choice([None, width + 3]))


def test_fork_without_enough_pages_and_entries_that_are_none():
    table = [[3, 4, 5, -7], [-7] * 4, [-7] * 4, [6, -1, 99, 2 ** 31 - 1], [-7] * 4, [-7] * 4, [-7] * 4]
    kv = [40, 0, 0, 64, 0, 0, 0]
    parents = [-1, 0, 0, 3, 3, 3, 0]
    for lens in (None, [0, 40, 7, 0, 20, 33, 40]):
        for free, head in (([], None), ([9], None), ([9, 8], 1), ([9, 8], 7), ([9, -1, 55, 7], 1), ([9, 8, 1, 2], -4)):
            run_fork(parents, lens, kv, free, max(head, 0) if head is not None else None, table, 16, [0] * 12)
    # a negative head counts as zero: rows 1, 2 and 6 take a page each
    k, s, t = dev(kv), dev([0] * 12), dev(table)
    _, counts = fa.attn_paged_fork(dev(parents), k, dev([9, 8, 1]), t, 16, s, free_head=dev([-4]))
    assert counts.tolist() == [5, 3, 0, 0]


def test_fork_parents_out_of_range_and_lengths_past_the_table():
    table = [[1, 2], [3, 4], [-7, -7], [-7, -7]]
    run_fork([4, -2 ** 31, 2 ** 31 - 1, 0], None, [32, 5, 0, 0], [8, 9], None, table, 16, [0] * 10)
    run_fork([-1, -1, 0, 1], None, [2 ** 31 - 1, -5, 7, 7], [8, 9], None, table, 16, [0] * 10)
    run_fork([1, 2, 3, -1], None, [20, 20, 20, 20], [8, 9], None, table, 16, [0] * 10)   # a chain: only row 2 may
    run_fork([1, 0, 0, 1], None, [20, 20, 20, 20], [8, 9], None, table, 16, [0] * 10)    # a ring


# ------------------------------------------------------------------ free
def run_free(kv, keep, table, page, shares, free, head, stride=None):
    room, t = wide_table(table, stride)
    s, f = dev(shares), dev(free)
    counts = fa.attn_paged_free(dev(kv), dev(keep), t, page, s, f, dev([head]))
    ok()
    want = plain_free(kv, keep, table, page, shares, free, head)
    for name, a, b in zip(("shares", "free", "counts"), (s, f, counts), want):
        assert a.tolist() == b, name
    assert t.tolist() == table and (stride is None or (room[:, len(table[0]):] == 77).all())


@pytest.mark.parametrize("n,page,hi,spare", [(1, 16, 100, 0), (2, 1, 9, 5), (3, 16, 100, 9000), (64, 16, 900, 100),
                                             (300, 7, 500, 3), (1024, 16, 300, 70000), (2500, 16, 60, 1)])
@pytest.mark.parametrize("shared", [False, True])
def test_free(n, page, hi, spare, shared):
    rng = random.Random(n + page)
    width = hi // page + 3
    n_pages = n * (hi // page + 1) + spare
    kv, table, rest = random_rows(rng, n, page, hi, width, n_pages)
    shares = [0] * n_pages
    if shared:  # rows name pages of others too, and some counts say that there are more of them than there are
        for i in range(n):
            j = rng.randrange(n)
            m = rng.randint(0, min(kv[i], kv[j]) // page)
            table[i][:m] = table[j][:m]
        for row, x in zip(table, kv):
            for col in range(-(-x // page)):
                shares[row[col]] += 1
        shares = [max(x - 1, 0) + (rng.random() < 0.05) for x in shares]
    keep = [rng.choice([0, x, max(0, x - rng.randint(0, 20)), rng.randint(-5, hi + 5)]) for x in kv]
    taken = n_pages - len(rest)
    free = [-5] * taken + rest
    run_free(kv, keep, table, page, shares, free, taken, stride=rng.choice([None, width + 2]))


def test_free_lists_without_room_and_heads_out_of_range():
    table = [[5, 1, 3], [7, 2, -7]]
    for head in (-3, 0, 1, 2, 4, 5, 9):
        run_free([48, 20], [0, 0], table, 16, [0] * 9, [11, 12, 13, 14, 15], head)


def test_free_entries_that_are_none_rows_named_twice_and_cuts():
    table = [[-1, 2 ** 31 - 1, 4, 9], [4, 4, 4, 4], [6, 7, 8, 0], [6, 7, 8, 1]]
    shares = [0, 0, 0, 0, 1, 0, 1, 1, 1, 0]
    run_free([64, 64, 64, 64], [0, 0, 0, 0], table, 16, shares, [-1] * 12, 12)       # 4 is named more often than counted
    run_free([64, 0, 64, 64], [10, 0, 40, 64], table, 16, shares, [-1] * 12, 12)     # cut inside a shared page
    run_free([64, 0, 64, 64], [64, 0, 40, 20], table, 16, shares, [-1] * 12, 12)     # both cut
    run_free([2 ** 31 - 1, -9, 70, 64], [-4, 3, 2 ** 31 - 1, 65], table, 16, shares, [-1] * 12, 12)


def test_free_is_the_same_in_every_run():
    n, page = 600, 16
    table = torch.randint(0, 3000, (n, 40), dtype=I32, device="cuda")
    kv, keep = torch.full((n,), 640, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
    outs = []
    for _ in range(5):
        shares, free = torch.full((3000,), 3, dtype=I32, device="cuda"), torch.zeros(3000, dtype=I32, device="cuda")
        counts = fa.attn_paged_free(kv, keep, table, page, shares, free, dev([3000]))
        outs.append((shares.tolist(), free.tolist(), counts.tolist()))
    ok()
    assert all(x == outs[0] for x in outs)


# ------------------------------------------------------------------ copy
def caches_of(kind, m, n_pages, page, H, x, dtype):
    def fresh(*shape):
        t = torch.randint(0, 256, (*shape, torch.empty((), dtype=dtype).element_size()), dtype=torch.uint8, device="cuda")
        return t.view(dtype).squeeze(-1)
    if kind == "tokens":
        return [fresh(n_pages, page, H, x) for _ in range(m)]
    if kind == "heads":
        return [fresh(n_pages, H, page, x).transpose(1, 2) for _ in range(m)]
    if kind == "wide":
        return list(fresh(n_pages, page, H, m * x).split(x, dim=-1))
    return list(fresh(n_pages, m, page, H, x).unbind(1))


@pytest.mark.parametrize("kind", ["tokens", "heads", "wide", "turns"])
@pytest.mark.parametrize("m,n_pages,page,H,x,dtype", [
    (1, 9, 16, 8, 128, torch.bfloat16), (2, 30, 16, 2, 64, torch.float16), (2, 12, 7, 3, 4, torch.uint8),
    (3, 10, 48, 1, 8, torch.uint8), (2, 40, 1, 5, 64, torch.uint8), (2, 11, 256, 8, 256, torch.bfloat16),
    (300, 8, 4, 2, 16, torch.uint8), (2, 9, 33, 4, 12, torch.uint8), (2, 9, 20, 4, 10, torch.float32)])
def test_copy(kind, m, n_pages, page, H, x, dtype):
    rng = random.Random(m + page)
    caches = caches_of(kind, m, n_pages, page, H, x, dtype)
    pages = rng.sample(range(n_pages), n_pages)
    src, dst = pages[:n_pages // 2], pages[n_pages // 2:]
    copies = [[rng.choice(src), d, rng.choice([1, page, rng.randint(1, page), page + 5])] for d in dst[:-1]]
    copies += [[-1, dst[-1], 3], [src[0], -1, 3], [src[0], n_pages, 3], [n_pages, dst[-1], 3], [src[0], dst[-1], 0],
               [src[0], dst[-1], -2], [src[0], src[0], 3], [2 ** 31 - 1, dst[-1], 3]]
    rng.shuffle(copies)
    want = [c.clone() for c in caches]
    for a, b, r in copies:
        if 0 <= a < n_pages and 0 <= b < n_pages and r > 0:
            for w in want:
                w[b, :r] = w[a, :r]
    fa.attn_paged_copy(dev(copies), caches)
    ok()
    for c, w in zip(caches, want):
        assert torch.equal(c.contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))


def test_copy_many_entries_and_two_layouts():
    n_pages, page, H = 3001, 4, 2
    caches = caches_of("heads", 2, n_pages, page, H, 64, torch.uint8) + caches_of("tokens", 2, n_pages, page, H, 8, torch.uint8)
    src = torch.randint(0, 1500, (1500,), dtype=I32, device="cuda")
    copies = torch.stack([src, torch.arange(1500, 3000, dtype=I32, device="cuda"),
                          torch.randint(1, 5, (1500,), dtype=I32, device="cuda")], 1)
    copies = torch.cat([copies, torch.full((2600, 3), -1, dtype=I32, device="cuda")])[torch.randperm(4100, device="cuda")]
    want = []
    for c in caches:
        mine = (torch.arange(page, device="cuda") < copies[:, 2:3])[:, :, None, None] & (copies[:, 0] >= 0)[:, None, None, None]
        a, b = (copies[:, i].long().clamp(min=0) for i in (0, 1))
        b = torch.where(copies[:, 0] >= 0, b, 3000)
        want.append(c.clone().index_copy_(0, b, torch.where(mine, c[a], c[b])))
    fa.attn_paged_copy(copies, caches)
    ok()
    assert all(torch.equal(c, w) for c, w in zip(caches, want))


def test_copy_offsets_past_32_bits():
    n_pages, page, H, x = 40000, 64, 8, 256
    big = torch.zeros(n_pages, page, H, x, dtype=torch.uint8, device="cuda")  # 5.2 GB
    big[3] = 5
    big[n_pages - 2] = torch.arange(256, device="cuda").to(torch.uint8)
    fa.attn_paged_copy(dev([[n_pages - 2, n_pages - 1, 9], [3, n_pages - 7, 64], [n_pages - 2, 1, 1]]), [big])
    ok()
    assert torch.equal(big[n_pages - 1, :9], big[n_pages - 2, :9]) and (big[n_pages - 1, 9:] == 0).all()
    assert (big[n_pages - 7] == 5).all() and torch.equal(big[1, :1], big[n_pages - 2, :1]) and (big[1, 1:] == 0).all()


# ------------------------------------------------------------------ a run of them
def test_calls_on_streams_and_from_a_graph():
    rng = random.Random(5)
    kv, table, rest = random_rows(rng, 30, 16, 200, 20, 600)
    parents = [rng.randrange(30) if x == 0 else -1 for x in kv]
    shares = [0] * 600
    cache = torch.randn(600, 16, 2, 64, device="cuda").to(torch.bfloat16)
    start = [dev(kv), dev(table), dev(shares)]
    k, t, s = (x.clone() for x in start)
    p, f, keep, head = dev(parents), dev([-1] * 50 + rest), dev([0] * 30), dev([50])
    copies, counts = torch.empty((30, 3), dtype=I32, device="cuda"), torch.empty(4, dtype=I32, device="cuda")
    freed = torch.empty(4, dtype=I32, device="cuda")

    def step(stream=None):
        fa.attn_paged_fork(p, k, f, t, 16, s, free_head=head, copies=copies, counts=counts, stream=stream)
        fa.attn_paged_copy(copies, [cache], stream=stream)
        fa.attn_paged_free(k, keep, t, 16, s, f, counts[1:2], counts=freed, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    ok()
    first = [x.clone() for x in (k, t, s, f, copies, counts, freed, cache)]
    free = [-1] * 50 + rest
    wk, wt, ws, wc, wn = plain_fork(parents, None, kv, free, 50, table, 16, shares)
    us, uf, un = plain_free(wk, [0] * 30, wt, 16, ws, free, wn[1])
    assert [x.tolist() for x in first[:7]] == [wk, wt, us, uf, wc, wn, un]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x, y in zip((k, t, s), start):
            x.copy_(y)
        f.copy_(dev(free))
        graph.replay()
    ok()
    for x, y in zip((k, t, s, f, copies, counts, freed, cache), first):
        assert torch.equal(x, y)
