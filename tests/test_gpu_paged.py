"""The paged key/value cache on the GPU: tables, cache write and attention against
plain 64-bit implementations, and the three of them in a run."""
import random

import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged_ref import Batch, check, plain_tables
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from attention_forward_11_gb300 import build
    build.build()
    fa.load_library()


def ok():
    assert fa.attn_check_device_status() == fa.ATTN_OK


# ------------------------------------------------------------------ tables
def run_tables(ctx, new, free, head, width, page, max_tokens, stride=None, seed=0):
    """Both implementations on rows that hold old pages where there are some and -7 elsewhere."""
    rng = random.Random(seed)
    n = len(ctx)
    table = [[rng.randrange(1 << 20) if c < -(-max(x, 0) // page) else -7 for c in range(width)] for x in ctx]
    wide = torch.full((n, stride or width), 77, dtype=I32, device="cuda")
    wide[:, :width] = torch.tensor(table, dtype=I32)
    got_table = wide[:, :width]
    dev = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    out = fa.attn_paged_tables(dev(ctx), dev(new), dev(free), got_table, page, max_tokens,
                               free_head=None if head is None else dev([head]))
    ok()
    want = plain_tables(ctx, new, free, head or 0, table, page, max_tokens)
    for name, a, b in zip(("table", "cu", "kv", "slots", "counts"), (got_table, *out), want):
        assert a.tolist() == b, name
    if stride:
        assert (wide[:, width:] == 77).all()


@pytest.mark.parametrize("n,page,hi,new_hi", [(1, 16, 0, 1), (1, 1, 5, 4), (3, 16, 100, 1), (64, 16, 900, 1),
                                              (70, 48, 500, 90), (1000, 64, 3000, 40), (1024, 32, 60, 3),
                                              (1025, 128, 2000, 5), (2500, 16, 200, 30)])
def test_tables(n, page, hi, new_hi):
    rng = random.Random(n + page)
    ctx = [rng.randint(0, hi) for _ in range(n)]
    new = [rng.choice([0, 1, rng.randint(0, new_hi)]) for _ in range(n)]
    free = rng.sample(range(1 << 24), n * (new_hi // page + 2))
    run_tables(ctx, new, free, rng.choice([None, 3]), (hi + new_hi) // page + 3, page, sum(new) + 37, seed=n)


def test_tables_lengths_at_the_edges():
    # nothing new, nothing cached, exactly full pages, negative lengths, a pad row
    run_tables([0, 16, 15, 17, 32, -4, 5, 0], [0, 16, 1, 0, 1, 3, -2, 1], list(range(50, 90)), 2, 8, 16, 30, stride=11)


def test_tables_without_enough_pages():
    run_tables([5, 0, 20], [40, 30, 1], [9, 8, 7], None, 8, 16, 71)   # the list runs out inside a sequence
    run_tables([5, 0, 20], [40, 30, 40], [9, 8, 7], 5, 8, 16, 200)    # it starts past its end
    run_tables([5, 0, 20], [40, 30, 40], [], None, 8, 16, 200)        # there is none


def test_tables_rows_too_narrow_and_slots_cut():
    run_tables([5, 70, 20], [40, 30, 100], list(range(20)), None, 3, 16, 200)
    run_tables([5, 70, 20], [40, 30, 100], list(range(20)), None, 9, 16, 33)
    run_tables([5], [2000], list(range(200)), None, 200, 16, 1)


def test_tables_old_pages_that_are_none():
    table = torch.tensor([[4, -1, 9, -1]], dtype=I32, device="cuda")
    one = lambda x: torch.tensor([x], dtype=I32, device="cuda")  # noqa: E731
    _, _, slots, _ = fa.attn_paged_tables(one(24), one(10), one(3), table, 16, 12)
    # columns 0 and 1 are the cached tokens' (24 of them), column 2 is new and takes page 3
    assert table.tolist() == [[4, -1, 3, -1]] and slots.tolist() == [-1] * 8 + [48, 49, -1, -1]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("T,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 1, BF, "tokens"), (1, 8, 128, 16, HF, "heads"), (37, 2, 64, 48, BF, "turns"),
    (300, 8, 128, 16, BF, "tokens"), (129, 3, 256, 7, HF, "heads"), (5, 40, 128, 32, BF, "turns"),
    (2000, 1, 128, 128, HF, "tokens")])
@pytest.mark.parametrize("fused", [False, True])
def test_append(T, Hkv, D, page, dtype, layout, fused):
    g = torch.Generator(device="cuda").manual_seed(T)
    b = Batch([(T + 3 * page, 0)], Hkv, Hkv, D, page, dtype, layout=layout, stale=2.5, seed=T)
    n_slots = b.n_pages * page
    if fused:
        x = torch.randn(T, 3 * Hkv + 1, D, dtype=dtype, device="cuda", generator=g)
        k, v = x[:, 1:1 + Hkv], x[:, 1 + 2 * Hkv:]
    else:
        k, v = (torch.randn(T, Hkv, D, dtype=dtype, device="cuda", generator=g) for _ in range(2))
    slots = torch.randperm(n_slots, device="cuda", generator=g)[:T]
    if T > 4:  # rows that are skipped: no slot, one past the end, far away
        slots[1], slots[2], slots[3], slots[4] = -1, n_slots, 1 << 45, -(1 << 40)
    want = [c.clone() for c in (b.k_cache, b.v_cache)]
    for t, x in enumerate(slots.tolist()):
        if 0 <= x < n_slots:
            want[0][x // page, x % page] = k[t]
            want[1][x // page, x % page] = v[t]
    fa.attn_paged_append(k, v, slots, b.k_cache, b.v_cache)
    ok()
    assert torch.equal(b.k_cache, want[0]) and torch.equal(b.v_cache, want[1])


def test_append_same_slot_twice_holds_one_of_the_rows():
    b = Batch([(32, 0)], 2, 2, 64, 16, stale=0.0)
    k = torch.stack([torch.full((2, 64), float(i + 1), dtype=BF, device="cuda") for i in range(2)])
    fa.attn_paged_append(k, k, torch.tensor([5, 5], device="cuda"), b.k_cache, b.v_cache)
    ok()
    for c in (b.k_cache, b.v_cache):
        assert ((c[0, 5] == 1) | (c[0, 5] == 2)).all()


# ------------------------------------------------------------------ attention
def run_fwd(b, **kw):
    """o and lse of a call whose outputs were filled with a sentinel."""
    a = b.on_gpu()
    o = torch.full((b.q.shape[0], b.Hq, b.D), 9.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.Hq, b.q.shape[0]), 9.0, dtype=torch.float32, device="cuda")
    kw = {"max_q_len": max(max(n for _, n in b.lens), 1), **kw}
    fa.attn_paged_fwd(**a, causal=b.causal, scale=b.scale, o=o, lse=lse, **kw)
    ok()
    return o, lse


DECODE = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (129, 1), (500, 1), (1037, 1)]
VERIFY = [(5, 5), (40, 3), (700, 5), (129, 1), (64, 4)]
CHUNKS = [(1, 1), (300, 300), (513, 200), (129, 129), (1000, 37), (260, 130), (70, 70)]
MIXED = [(900, 1), (333, 333), (77, 1), (2, 2), (1500, 150), (128, 1)]


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 16, BF, "tokens"), (8, 1, 128, 16, BF, "heads"), (4, 2, 128, 32, HF, "turns"),
    (6, 2, 64, 48, HF, "tokens"), (14, 2, 128, 64, BF, "heads"), (16, 1, 64, 128, BF, "tokens"),
    (5, 1, 256, 16, BF, "turns"), (8, 4, 128, 1, BF, "tokens"), (3, 3, 64, 7, HF, "heads"), (2, 1, 128, 1024, BF, "tokens"),
    (23, 1, 128, 16, BF, "tokens"), (46, 2, 64, 80, HF, "turns")])
@pytest.mark.parametrize("name", ["decode", "verify", "chunks", "mixed"])
def test_fwd(name, Hq, Hkv, D, page, dtype, layout):
    lens = {"decode": DECODE, "verify": VERIFY, "chunks": CHUNKS, "mixed": MIXED}[name]
    b = Batch(lens, Hq, Hkv, D, page, dtype, layout=layout, pad_rows=3, seed=len(name) + Hq)
    o, lse = run_fwd(b)
    check(b, o, lse, untouched=9.0)


@pytest.mark.parametrize("Hq,Hkv,D,page,layout", [
    (4, 2, 128, 16, "wide"), (4, 2, 64, 64, "wide"), (4, 2, 128, 128, "wide"),   # heads 2 D apart
    (47, 1, 64, 7, "tokens"), (80, 2, 128, 1, "heads"),                             # groups past a block's rows
    (160, 1, 64, 16, "tokens"), (140, 1, 128, 32, "turns"), (50, 1, 256, 16, "tokens")])
@pytest.mark.parametrize("lens", [[(130, 1), (17, 1), (400, 1)], [(200, 70), (33, 5), (300, 1)]], ids=["decode", "chunk"])
def test_fwd_wide_rows_and_groups(lens, Hq, Hkv, D, page, layout):
    b = Batch(lens, Hq, Hkv, D, page, layout=layout, pad_rows=1, seed=Hq)
    check(b, *run_fwd(b), untouched=9.0)


@pytest.mark.parametrize("n", [257, 700])
@pytest.mark.parametrize("kind", ["decode", "chunks", "mixed"])
def test_fwd_many_sequences(n, kind):
    """More sequences than a block has threads: the lengths are read in several steps."""
    rng = random.Random(n)
    lens = []
    for i in range(n):
        q = {"decode": 1, "chunks": rng.randint(1, 40), "mixed": 200 if i % 97 == 5 else 1}[kind]
        q = 0 if rng.random() < 0.1 else q
        lens.append((q + rng.randint(0, 60), q))
    b = Batch(lens, 4, 2, 64, 16, seed=n)
    check(b, *run_fwd(b))
    if kind == "decode":
        b = Batch(lens, 2, 1, 256, 16, seed=n)
        check(b, *run_fwd(b))


@pytest.mark.parametrize("D,group", [(64, 4), (128, 3)])
def test_fwd_one_chunk_among_single_tokens(D, group):
    """Batches whose single tokens and chunks are different kernels' (many of the former)."""
    lens = [(1 + 7 * i, 1) for i in range(150)]
    lens[40], lens[90], lens[91] = (700, 300), (2, 2), (40, 0)
    b = Batch(lens, 2 * group, 2, D, 16, pad_rows=2, seed=D)
    for max_q in (300, 10 ** 6, 60):
        check(b, *run_fwd(b, max_q_len=max_q), untouched=9.0)


def test_fwd_one_long_sequence_among_many():
    """Shares that cut one unit many times and take others whole."""
    lens = [(30000, 1)] + [(rng, 1) for rng in range(1, 200)]
    b = Batch(lens, 4, 1, 64, 16, seed=3)
    check(b, *run_fwd(b))
    lens = [(30000, 40), (3, 3)] + [(100 + i, 50) for i in range(30)]
    b = Batch(lens, 2, 1, 64, 16, seed=3)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("lens,max_q", [([(20000, 1), (9000, 1), (40, 1)], 1), ([(20000, 100), (300, 1), (8000, 1)], 100)],
                         ids=["rows", "mixed"])
def test_fwd_workspace_contents_do_not_matter(lens, max_q):
    b = Batch(lens, 8, 1, 128, 16, seed=30)
    a = b.on_gpu()
    size = fa.attn_paged_fwd_workspace_size(b.T, max_q, 8, 1, 128, 16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = None
    g = torch.Generator(device="cuda").manual_seed(1)
    for fill in ("zero", "ones", "random", "nan", "as left", "as left"):
        if fill == "ones":
            ws.fill_(255)
        elif fill == "random":
            ws.copy_(torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda", generator=g))
        elif fill == "nan":
            ws[:size // 4 * 4].view(torch.float32).fill_(float("nan"))
        o, lse = fa.attn_paged_fwd(**a, max_q_len=max_q, workspace=ws)
        ok()
        if first is None:
            first = (o, lse)
            check(b, o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), fill


def test_two_graphs_that_share_a_workspace():
    """Replayed one after the other, in any order, each many times."""
    bs = [Batch([(20000, 1), (37, 1)], 8, 1, 128, 16, seed=31), Batch([(9000, 60), (500, 1)], 8, 1, 128, 16, seed=32)]
    size = max(fa.attn_paged_fwd_workspace_size(b.T, 60, 8, 1, 128, 16) for b in bs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for b, max_q in zip(bs, (1, 60)):
        a = b.on_gpu()
        o = torch.empty_like(a["q"])
        lse = torch.empty((8, b.q.shape[0]), dtype=torch.float32, device="cuda")
        fa.attn_paged_fwd(**a, max_q_len=max_q, o=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.attn_paged_fwd(**a, max_q_len=max_q, o=o, lse=lse, workspace=ws)
        graphs.append((g, a))
        outs.append((o, lse))
    for i in (0, 0, 1, 0, 1, 1, 0):
        outs[i][0].fill_(9.0)
        graphs[i][0].replay()
    ok()
    for b, (o, lse) in zip(bs, outs):
        check(b, o, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", ["verify", "mixed"])
def test_fwd_every_key_visible(name, D):
    b = Batch(VERIFY if name == "verify" else MIXED, 4, 2, D, 16, causal=0, seed=D)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D,group", [(64, 1), (128, 4), (256, 2)])
def test_fwd_rows_without_keys_and_empty_sequences(D, group):
    # more rows than keys, no key at all, no row, and rows of no sequence at the end
    lens = [(0, 1), (3, 7), (0, 0), (40, 0), (0, 130), (100, 300), (5, 1)]
    b = Batch(lens, 2 * group, 2, D, 16, pad_rows=5, seed=2)
    check(b, *run_fwd(b), untouched=9.0)
    b = Batch([(0, 0), (0, 0)], 2 * group, 2, D, 16, pad_rows=5, seed=2)
    check(b, *run_fwd(b), untouched=9.0)


@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
@pytest.mark.parametrize("max_q", [1, 3, 100000])
def test_fwd_is_right_for_any_max_q_len(lens, max_q):
    b = Batch(lens, 8, 2, 128, 16, seed=4)
    a = b.on_gpu()
    o, lse = fa.attn_paged_fwd(**a, max_q_len=max_q, causal=1, scale=b.scale)
    ok()
    check(b, o, lse)
    o2, lse2 = fa.attn_paged_fwd(**a, max_q_len=max_q, causal=1, scale=b.scale)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("stale", [float("nan"), float("inf"), -3.0e38])
@pytest.mark.parametrize("lens", [[(33, 1), (130, 1)], [(200, 150), (33, 20)]], ids=["rows", "tiles"])
def test_fwd_stale_rows_have_no_influence(lens, stale):
    b = Batch(lens, 4, 1, 128, 64, stale=stale, seed=1)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "n_pages"])
@pytest.mark.parametrize("lens", [[(100, 1), (300, 1)], [(100, 40), (300, 200)]], ids=["rows", "tiles"])
@pytest.mark.parametrize("page", [16, 32, 100])
def test_fwd_entries_that_name_no_page(lens, bad, page):
    b = Batch(lens, 4, 2, 64, page, seed=7)
    where = [(0, 0), (1, 1), (1, 2)]
    for s, col in where:
        b.table[s, col] = b.n_pages if bad == "n_pages" else bad
    o, lse = run_fwd(b)
    check(b, o, lse, bad_pages=where)


def test_fwd_no_page_at_all():
    b = Batch([(100, 1), (300, 150)], 4, 2, 64, 16, seed=7)
    b.table[:] = -1
    o, lse = run_fwd(b)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_fwd_lengths_that_are_out_of_range():
    """Ranges of rows outside q and keys past the table are cut, not followed."""
    b = Batch([(64, 2), (64, 3)], 4, 2, 64, 16, extra_cols=0, seed=9)
    a = b.on_gpu()
    a["kv_lens"] = torch.tensor([2 ** 31 - 1, -9], dtype=I32, device="cuda")
    a["cu_q"] = torch.tensor([-5, 2, 2 ** 31 - 1], dtype=I32, device="cuda")
    for max_q in (1, 1000):
        o, lse = fa.attn_paged_fwd(**a, max_q_len=max_q, causal=1, scale=b.scale)
        ok()
        want, wl, tol, tl = Batch([(64, 2), (64, 3)], 4, 2, 64, 16, extra_cols=0, seed=9).reference()
        assert (np.abs(o.double().cpu().numpy() - want)[:2] <= tol[:2]).all()
        assert (o[2:] == 0).all() and torch.isneginf(lse[:, 2:]).all()
    a["cu_q"] = torch.tensor([4, 1, 0], dtype=I32, device="cuda")  # falling: no rows
    o = torch.full_like(a["q"], 9.0)
    fa.attn_paged_fwd(**a, max_q_len=1, o=o)
    ok()
    assert (o == 9.0).all()


def test_fwd_sharp_logits_and_nan_in_a_seen_key():
    b = Batch(MIXED, 4, 2, 128, 16, seed=11, q_sigma=8.0)
    check(b, *run_fwd(b))
    b = Batch([(50, 1), (60, 1)], 4, 2, 128, 64, seed=12)
    b.k_cache[b.table[0, 0], 3] = float("nan")
    for max_q in (1, 1000):
        o, lse = run_fwd(b, max_q_len=max_q)
        assert torch.isnan(o[0].float()).all() and torch.isnan(lse[:, 0]).all()
        assert torch.isfinite(o[1].float()).all()


@pytest.mark.parametrize("lens", [[(20000, 1)], [(20000, 1), (31, 1), (9000, 3)], [(17000, 20)], [(17000, 64), (100, 1)]],
                         ids=["one", "rows", "short_chunk", "chunk"])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 64), (8, 1, 128), (4, 1, 256)])
def test_fwd_long_caches(lens, Hq, Hkv, D):
    b = Batch(lens, Hq, Hkv, D, 16, seed=5)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D", [64, 128])
def test_fwd_wide_rows_of_a_fused_projection(D):
    b = Batch(MIXED, 8, 2, D, 16, seed=6)
    a = b.on_gpu()
    x = torch.randn(b.T, 12, D, device="cuda").to(BF)
    x[:, :8] = a["q"]
    a["q"] = x[:, :8]
    wide = torch.full((len(b.lens), b.table.shape[1] + 5), 2 ** 30, dtype=I32, device="cuda")
    wide[:, :b.table.shape[1]] = a["block_table"]
    a["block_table"] = wide[:, :b.table.shape[1]]
    for max_q in (1, 1000):
        check(b, *fa.attn_paged_fwd(**a, max_q_len=max_q, causal=1))
        ok()


@pytest.mark.parametrize("shift", [-60.0, -17.3, 40.0])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, HF), (128, BF), (256, HF)])
@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
def test_fwd_logits_far_from_zero(lens, D, dtype, shift):
    """Weights are relative to the row's own maximum, however far below zero that is: fp16
    weights relative to anything higher would vanish."""
    b = Batch(lens, 4, 2, D, 16, dtype, seed=15, shift=shift)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("scale", [0.01, 0.7])
@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF), (256, HF)])
def test_fwd_arguments_left_out_and_other_scales(D, dtype, scale):
    b = Batch(MIXED, 4, 2, D, 32, dtype, seed=14)
    a = b.on_gpu()
    b.scale = scale
    o, lse = fa.attn_paged_fwd(**a, scale=scale)                  # max_q_len left out
    ok()
    check(b, o, lse)
    o2, none = fa.attn_paged_fwd(**a, scale=scale, want_lse=False)
    ok()
    assert none is None and torch.equal(o, o2)
    big = torch.empty(64 << 20, dtype=torch.float32, device="cuda")  # more workspace than needed, another type
    o3, lse3 = fa.attn_paged_fwd(**a, scale=scale, workspace=big)
    ok()
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_past_32_bits(D):
    """A cache of more than 2^32 bytes and 2^31 elements whose used pages are the last ones."""
    page, Hkv = 64, 8
    first = (5 << 29) // (page * Hkv * D)  # 2.7e9 elements before the first page in use
    b = Batch([(200, 1), (513, 70)], 16, Hkv, D, page, first_page=first, seed=8)
    assert b.k_cache.numel() > 1 << 31
    for max_q in (1, 70):
        check(b, *run_fwd(b, max_q_len=max_q))
    rows = torch.randn(3, Hkv, D, device="cuda").to(BF)
    slots = torch.tensor([b.n_pages * page - 1, first * page, 5], device="cuda")
    fa.attn_paged_append(rows, rows, slots, b.k_cache, b.v_cache)
    ok()
    assert torch.equal(b.k_cache[-1, -1], rows[0]) and torch.equal(b.v_cache[first, 0], rows[1])
    assert torch.equal(b.v_cache[0, 5], rows[2])


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_fwd_writes_inside_its_buffers(lens, D):
    b = Batch(lens, 8, 2, D, 16, seed=13)
    a = b.on_gpu()
    max_q = max(n for _, n in lens)
    o, lse = Guarded((b.T, 8, D), BF), Guarded((8, b.T), torch.float32)
    size = fa.attn_paged_fwd_workspace_size(b.T, max_q, 8, 2, D, 16)
    ws = Guarded((max(size, 4),), torch.uint8)
    fa.attn_paged_fwd(**a, max_q_len=max_q, causal=1, scale=b.scale, o=o.t, lse=lse.t, workspace=ws.t)
    ok()
    assert o.guards_intact() and lse.guards_intact() and ws.guards_intact()
    assert o.fully_written() and lse.fully_written()
    check(b, o.t, lse.t)


def test_fwd_refuses_a_short_workspace_and_launches_nothing():
    b = Batch([(4000, 1)], 8, 2, 128, 16, seed=1)
    a = b.on_gpu()
    size = fa.attn_paged_fwd_workspace_size(b.T, 1, 8, 2, 128, 16)
    before = fa.attn_kernel_launches()
    if size:
        with pytest.raises(fa.AttnError) as e:
            fa.attn_paged_fwd(**a, max_q_len=1, workspace=torch.empty(size - 256, dtype=torch.uint8, device="cuda"))
        assert e.value.status == fa.ATTN_ERR_INVALID_ARG
    for over in (dict(q=a["q"].float()), dict(cu_q=a["cu_q"].long()), dict(kv_lens=a["kv_lens"].repeat(2)),
                 dict(block_table=a["block_table"].t()), dict(v_cache=a["v_cache"][:, :8]), dict(q=a["q"][:, :7]),
                 dict(o=torch.empty(1, 8, 128, device="cuda")), dict(lse=torch.empty(1, 8, device="cuda")),
                 dict(kv_lens=a["kv_lens"].cpu())):
        with pytest.raises(fa.AttnError):
            fa.attn_paged_fwd(**{**a, "max_q_len": 1, **over})
    assert fa.attn_kernel_launches() == before


# ------------------------------------------------------------------ a run of them
class Server:
    """Two-layer cache of growing sequences; what the GPU holds is compared with dense copies."""

    def __init__(self, n, Hq, Hkv, D, page, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.Hq, self.Hkv, self.D, self.page = n, Hq, Hkv, D, page
        self.n_pages = 400
        self.cache = torch.full((2, self.n_pages, 2, page, Hkv, D), float("nan"), dtype=BF, device="cuda")
        self.table = torch.full((n, 64), -1, dtype=I32, device="cuda")
        self.free = torch.randperm(self.n_pages, device="cuda", generator=self.g, dtype=I32)
        self.head = torch.zeros(1, dtype=I32, device="cuda")
        self.ctx = torch.zeros(n, dtype=I32, device="cuda")
        self.dense = [[[] for _ in range(n)] for _ in range(2)]

    def step(self, new_lens, qkv, new, cap, max_q):
        """One step on the GPU, without the host: all layers read the step's own tables."""
        cu, kv, slots, counts = fa.attn_paged_tables(self.ctx, new_lens, self.free, self.table, self.page, cap,
                                                     free_head=self.head)
        outs = []
        for layer in range(2):
            x = qkv[layer]
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
            kc, vc = self.cache[layer, :, 0], self.cache[layer, :, 1]
            fa.attn_paged_append(k, v, slots, kc, vc)
            outs.append(fa.attn_paged_fwd(q, kc, vc, self.table, cu, kv, max_q_len=max_q))
        self.ctx.copy_(kv)
        self.head.copy_(counts[1:2])
        return outs

    def compare(self, new, qkv, outs):
        at = 0
        for s, x in enumerate(new):
            for layer in range(2):
                rows = qkv[layer][at:at + x]
                self.dense[layer][s].append(rows[:, self.Hq:])
                if x == 0:
                    continue
                kv = torch.cat(self.dense[layer][s])
                b = Batch([(kv.shape[0], x)], self.Hq, self.Hkv, self.D, self.page, device="cpu")
                b.q = rows[:, :self.Hq].cpu()
                b.dense = [(kv[:, :self.Hkv].cpu(), kv[:, self.Hkv:].cpu())]
                o, lse = outs[layer]
                check(b, o[at:at + x], lse[:, at:at + x])
            at += x


STEPS = [[40, 0, 7, 130], [1, 33, 1, 1], [1, 1, 1, 0], [5, 1, 1, 200], [1, 1, 1, 1]]


def test_steps_of_a_server():
    sv = Server(4, 4, 2, 64, 16)
    for new in STEPS:
        cap = sum(new) + 4
        qkv = [torch.randn(cap, 8, 64, device="cuda", generator=sv.g).to(BF) for _ in range(2)]
        outs = sv.step(torch.tensor(new, dtype=I32, device="cuda"), qkv, new, cap, max(new))
        ok()
        sv.compare(new, qkv, outs)


@pytest.mark.parametrize("max_q", [1, 200])
def test_steps_replayed_from_a_graph(max_q):
    """One captured step, replayed with other lengths, tables and rows."""
    sv = Server(4, 4, 2, 64, 16, seed=1)
    cap = 340
    qkv = [torch.zeros(cap, 8, 64, dtype=BF, device="cuda") for _ in range(2)]
    new_lens = torch.zeros(4, dtype=I32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.step(new_lens, qkv, None, cap, max_q)  # nothing new: changes nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = sv.step(new_lens, qkv, None, cap, max_q)
    for new in STEPS:
        new_lens.copy_(torch.tensor(new, dtype=I32))
        for x in qkv:
            x.copy_(torch.randn(cap, 8, 64, device="cuda", generator=sv.g).to(BF))
        graph.replay()
        ok()
        sv.compare(new, [x.clone() for x in qkv], outs)


def test_two_streams_at_once():
    """Two batches on two streams, each call with its own workspace, interleaved."""
    bs = [Batch(DECODE, 8, 2, 128, 16, seed=20), Batch(CHUNKS, 8, 2, 128, 16, seed=21)]
    streams = [torch.cuda.Stream() for _ in bs]
    ins = [b.on_gpu() for b in bs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for i, b in enumerate(bs):
            outs[i].append(fa.attn_paged_fwd(**ins[i], max_q_len=max(n for _, n in b.lens), stream=streams[i]))
    torch.cuda.synchronize()
    ok()
    for i, b in enumerate(bs):
        for o, lse in outs[i]:
            assert torch.equal(o, outs[i][0][0]) and torch.equal(lse, outs[i][0][1])
        check(b, *outs[i][0])


@pytest.mark.parametrize("kind", ["none", "zero", "stream", "handle"])
def test_streams_in_every_form(kind):
    """A stream as torch's object, as a handle, as the default stream's handle 0, or none; the
    calls allocate their outputs themselves, and another stream's allocations in between must
    not disturb them."""
    side = torch.cuda.Stream()
    stream = {"none": None, "zero": 0, "stream": side, "handle": side.cuda_stream}[kind]
    b = Batch([(9000, 1), (40, 1)], 8, 1, 64, 16, seed=40)
    a = b.on_gpu()
    torch.cuda.synchronize()
    for _ in range(3):
        o, lse = fa.attn_paged_fwd(**a, max_q_len=1, stream=stream)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # on the current stream
        del junk
    one = torch.ones(2, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    cu, kv, slots, counts = fa.attn_paged_tables(a["kv_lens"], one, torch.arange(8, dtype=I32, device="cuda") + 9000,
                                                 a["block_table"], 16, 4, stream=stream)
    k = torch.randn(4, 1, 64, device="cuda").to(BF)
    torch.cuda.synchronize()
    fa.attn_paged_append(k, k, slots, b.k_cache, b.v_cache, stream=stream)
    torch.cuda.synchronize()
    ok()
    check(b, o, lse)
    assert cu.tolist() == [0, 1, 2] and kv.tolist() == [9001, 41] and counts.tolist()[0] == 2
    col = 40 // 16
    assert slots.tolist()[1] == int(a["block_table"][1, col]) * 16 + 8 and slots.tolist()[2:] == [-1, -1]


# ------------------------------------------------------------------ batches with many empty places
def padded(a, where, n):
    """The arguments of a batch whose sequence i stands at place where[i] of n, the others empty."""
    lens, kv = [0] * n, [0] * n
    table = torch.full((n, a["block_table"].shape[1]), -1, dtype=I32, device="cuda")
    cu = a["cu_q"].tolist()
    for i, w in enumerate(where):
        lens[w], kv[w] = cu[i + 1] - cu[i], int(a["kv_lens"][i])
        table[w] = a["block_table"][i]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=I32, device="cuda")
    return {**a, "block_table": table, "cu_q": cu, "kv_lens": torch.tensor(kv, dtype=I32, device="cuda")}


def device_us(call, calls=10):
    """Device time of one call among others, in a graph; the best of several replays."""
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(calls):
            call()
    times = []
    for _ in range(8):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        g.replay()
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]) * 1000 / calls)
    return min(times[1:])


@pytest.mark.parametrize("name,lens,Hq,Hkv,D,n,step,times", [
    # requests at the front of a large captured batch: their places are scanned (13 to 20 us), not walked (530 us)
    ("decode", [(1001, 1)] * 8, 32, 8, 128, 4096, 1, 4),
    ("decode", [(1001, 1)] * 8, 32, 8, 64, 4096, 1, 4),
    ("decode", [(300, 1)] * 8, 8, 4, 256, 4096, 1, 4),
    ("chunks", [(700, 64)] * 8, 32, 8, 128, 1024, 1, 2.5),
    # and spread over it: the walk from one to the next
    ("decode", [(2500 * (i + 1), 1) for i in range(12)], 4, 1, 128, 1024, 85, 1.5),
    ("mixed", [(200 + i, 300 if i % 7 == 3 else 1) for i in range(20)], 8, 2, 64, 1024, 51, 4),
])
def test_fwd_empty_places_of_a_batch(name, lens, Hq, Hkv, D, n, step, times):
    """The same bits as without them, in a time that does not grow with every empty place."""
    b = Batch(lens, Hq, Hkv, D, 16, seed=n + D)
    a = b.on_gpu()
    wide = padded(a, [i * step for i in range(len(lens))], n)
    max_q = max(q for _, q in lens)
    size = fa.attn_paged_fwd_workspace_size(b.T, max_q, Hq, Hkv, D, 16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs, took = [], []
    for args in (a, wide):
        o = torch.full_like(args["q"], 9.0)
        lse = torch.full((Hq, b.T), 9.0, device="cuda")
        took.append(device_us(lambda: fa.attn_paged_fwd(**args, max_q_len=max_q, o=o, lse=lse, workspace=ws)))
        ok()
        outs.append((o, lse))
        check(b, o, lse)
    if name != "mixed":  # there the empty places may choose other kernels
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert took[1] <= times * took[0], f"{took[0]:.1f} us, among {n} places {took[1]:.1f} us"


@pytest.mark.parametrize("D", [64, 128])
def test_fwd_empty_places_are_no_single_tokens(D):
    """A chunk and three tokens in 1024 places are no batch of many tokens: two kernels, the second
    joining the first one's pieces, as without the empty places."""
    lens = [(700, 512), (40, 1), (100, 1), (7, 1)]
    b = Batch(lens, 8, 2, D, 16, seed=D)
    a = padded(b.on_gpu(), [3, 200, 201, 1000], 1024)
    before = fa.attn_kernel_launches()
    o, lse = fa.attn_paged_fwd(**a, max_q_len=512)
    ok()
    assert fa.attn_kernel_launches() == before + 2
    check(b, o, lse)
    many = Batch([(700, 512)] + [(40, 1)] * 900, 2, 1, D, 16, seed=D)  # a batch of many tokens: three
    before = fa.attn_kernel_launches()
    o, lse = fa.attn_paged_fwd(**many.on_gpu(), max_q_len=512)
    ok()
    assert fa.attn_kernel_launches() == before + 3
    check(many, o, lse)


def test_fwd_units_of_a_few_more_keys_than_a_share_are_cut():
    """Head size 64: a chunk of 128 blocks of rows leaves no 24 of 152 SMs idle, which a chunk of 152
    blocks takes whole (0.86 of its time; with whole units 1.0)."""
    took = []
    for n in (608, 512):
        b = Batch([(32000 + n, n)], 64, 8, 64, 64, seed=n)
        a = b.on_gpu()
        ws = torch.empty(fa.attn_paged_fwd_workspace_size(n, n, 64, 8, 64, 64), dtype=torch.uint8, device="cuda")
        took.append(device_us(lambda: fa.attn_paged_fwd(**a, max_q_len=n, workspace=ws)))
        ok()
    assert took[1] <= 0.94 * took[0], f"608 rows {took[0]:.0f} us, 512 rows {took[1]:.0f} us"
