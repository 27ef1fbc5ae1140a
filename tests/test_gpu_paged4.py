"""The paged cache in 4 bits on the GPU: its write and attention over it against plain
implementations in 64 bits, and a server's steps with forked rows."""
import random

import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from paged4_ref import E2M1, E4M3, Batch4, decode, encode, place
from paged_ref import check
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


# ------------------------------------------------------------------ append
def run_append(k, v, slots, codes, scales, page, **units):
    n_slots = codes[0].shape[0] * page
    want = [x.cpu().numpy().copy() for x in (codes[0], scales[0], codes[1], scales[1])]
    for i, (x, unit) in enumerate(((k, units.get("k_unit", 1.0)), (v, units.get("v_unit", 1.0)))):
        c, b = encode(x.float().cpu().numpy(), np.float32(1.0 / np.float64(np.float32(unit))))
        for t, at in enumerate(slots.tolist()):
            if 0 <= at < n_slots:
                want[2 * i][at // page, at % page], want[2 * i + 1][at // page, at % page] = c[t], b[t]
    fa.attn_paged_coded_append(k, v, slots, codes[0], scales[0], codes[1], scales[1], **units)
    ok()
    for name, x, w in zip(("k_codes", "k_scales", "v_codes", "v_scales"), (codes[0], scales[0], codes[1], scales[1]), want):
        bad = np.argwhere(x.cpu().numpy() != w)
        assert len(bad) == 0, f"{name}: {len(bad)} of {w.size} bytes, first at {bad[0]}"


@pytest.mark.parametrize("T,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 1, BF, "tokens"), (1, 8, 128, 16, HF, "heads"), (37, 2, 64, 48, BF, "turns"),
    (300, 8, 128, 16, BF, "tokens"), (129, 3, 256, 7, HF, "heads"), (5, 40, 128, 32, BF, "wide"),
    (2000, 1, 128, 128, HF, "tokens"), (61, 17, 64, 24, BF, "heads"), (3, 130, 256, 16, HF, "turns")])
@pytest.mark.parametrize("fused", [False, True])
def test_append(T, Hkv, D, page, dtype, layout, fused):
    g = torch.Generator(device="cuda").manual_seed(T)
    n_pages = T // page + 5
    codes, scales = place((n_pages, page, Hkv, D // 2), layout, 0x5a), place((n_pages, page, Hkv, D // 16), layout, 0x5a)
    if fused:
        x = torch.randn(T, 3 * Hkv + 1, D, dtype=dtype, device="cuda", generator=g)
        k, v = x[:, 1:1 + Hkv], x[:, 1 + 2 * Hkv:]
    else:
        k, v = (torch.randn(T, Hkv, D, dtype=dtype, device="cuda", generator=g) for _ in range(2))
    slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:T]
    if T > 4:  # rows that are skipped: no slot, one past the end, far away
        slots[1], slots[2], slots[3], slots[4] = -1, n_pages * page, 1 << 45, -(1 << 40)
    units = {} if fused else dict(k_unit=0.04, v_unit=3.0)
    run_append(k, v, slots, codes, scales, page, **units)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_values_at_the_borders(dtype):
    """Quotients on and beside every border between two codes, for scales of every significand; blocks of
    zeros (of both signs), of the smallest and largest numbers, infinities and NaN."""
    rows = []
    rng = np.random.RandomState(3)
    for byte in list(range(1, 40)) + list(range(64, 127)):
        s = E4M3[byte]
        ties = s * np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
        beside = np.concatenate([ties, ties * (1 + 2.0 ** -8), ties * (1 - 2.0 ** -8), ties * (1 + 2.0 ** -11)])
        for _ in range(4):
            block = rng.choice(np.concatenate([beside, -beside, [0.0, -0.0]]), 16)
            block[rng.randint(16)] = 6 * s * rng.choice([-1, 1])
            rows.append(block)
        near = E4M3[byte:byte + 2].mean()  # the largest element's sixth between two scales
        for x in (near * 6, near * 6 * (1 + 2.0 ** -8), near * 6 * (1 - 2.0 ** -8)):
            block = rng.randn(16) * x / 4
            block = np.clip(block, -x, x)
            block[5] = x
            rows.append(block)
    tiny = float(torch.finfo(dtype).smallest_normal)
    big = float(torch.finfo(dtype).max)
    inf, nan = np.inf, np.nan
    for special in ([0.0, -0.0], [tiny, -tiny, 0.0], [tiny / 4, 0.0], [big, -big, 1.0], [inf, 1.0, -3.0], [-inf, 5.0],
                    [nan, 1.0, -2.0], [nan], [nan, inf, -inf], [2.0 ** -10 * 6, 1e-5], [2.0 ** -9 * 6, 0.01], [1e-6, -1e-7],
                    [2688.0, -2688.0], [2700.0, 3.0], [3e4, -2000.0]):
        rows.append(rng.choice(special, 16))
        rows[-1][0] = special[0]
    while len(rows) % 8:
        rows.append(rng.randn(16))
    x = torch.tensor(np.stack(rows).reshape(-1, 1, 128), device="cuda").to(dtype)
    y = x.flip(0).contiguous()
    T = x.shape[0]
    codes, scales = place((T, 1, 1, 64), "tokens", 0x5a), place((T, 1, 1, 8), "tokens", 0x5a)
    for units in ({}, dict(k_unit=0.3, v_unit=7.0), dict(k_unit=1e-30, v_unit=1e30), dict(k_unit=2.0 ** -100, v_unit=2.0 ** 100)):
        run_append(x, y, torch.randperm(T, device="cuda"), codes, scales, 1, **units)


def test_append_same_slot_twice_holds_bytes_of_either():
    k = torch.stack([torch.full((2, 64), float(i + 1), dtype=BF, device="cuda") for i in range(2)])
    codes, scales = place((2, 16, 2, 32), "tokens", 0), place((2, 16, 2, 4), "tokens", 0)
    fa.attn_paged_coded_append(k, k, torch.tensor([5, 5], device="cuda"), codes[0], scales[0], codes[1], scales[1])
    ok()
    either = [encode(k[i].float().cpu().numpy(), 1.0) for i in range(2)]
    for c, s in zip(codes, scales):
        assert ((c[0, 5].cpu().numpy() == either[0][0]) | (c[0, 5].cpu().numpy() == either[1][0])).all()
        assert ((s[0, 5].cpu().numpy() == either[0][1]) | (s[0, 5].cpu().numpy() == either[1][1])).all()


# ------------------------------------------------------------------ attention
def run_fwd(b, **kw):
    """o and lse of a call whose outputs were filled with a sentinel."""
    a = b.on_gpu()
    o = torch.full((b.q.shape[0], b.Hq, b.D), 9.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.Hq, b.q.shape[0]), 9.0, dtype=torch.float32, device="cuda")
    kw = {"max_q_len": max(max(n for _, n in b.lens), 1), **kw}
    fa.attn_paged_coded_fwd(**a, causal=b.causal, scale=b.scale, k_unit=b.k_unit, v_unit=b.v_unit, o=o, lse=lse, **kw)
    ok()
    return o, lse


DECODE = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (129, 1), (500, 1), (1037, 1)]
VERIFY = [(5, 5), (40, 3), (700, 5), (129, 1), (64, 4)]
CHUNKS = [(1, 1), (300, 300), (513, 200), (129, 129), (1000, 37), (260, 130), (70, 70)]
MIXED = [(900, 1), (333, 333), (77, 1), (2, 2), (1500, 150), (128, 1)]


def test_fwd_smallest():
    """Every element of a few keys on its own: an order that K and Q, or P and V, do not share shows here."""
    for D in (64, 128, 256):
        for kv in (1, 2, 16, 31):
            b = Batch4([(kv, 1)], 1, 1, D, 16, HF, seed=D + kv)
            check(b, *run_fwd(b))


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,layout", [
    (1, 1, 64, 16, BF, "tokens"), (8, 1, 128, 16, BF, "heads"), (4, 2, 128, 32, HF, "turns"),
    (6, 2, 64, 48, HF, "tokens"), (14, 2, 128, 64, BF, "heads"), (16, 1, 64, 128, BF, "tokens"),
    (5, 1, 256, 16, BF, "turns"), (8, 4, 128, 1, BF, "tokens"), (3, 3, 64, 7, HF, "heads"), (2, 1, 128, 1024, BF, "wide"),
    (23, 1, 128, 16, BF, "tokens"), (46, 2, 64, 80, HF, "turns"), (9, 1, 256, 24, HF, "wide")])
@pytest.mark.parametrize("name", ["decode", "verify", "chunks", "mixed"])
def test_fwd(name, Hq, Hkv, D, page, dtype, layout):
    lens = {"decode": DECODE, "verify": VERIFY, "chunks": CHUNKS, "mixed": MIXED}[name]
    b = Batch4(lens, Hq, Hkv, D, page, dtype, layout=layout, pad_rows=3, seed=len(name) + Hq)
    o, lse = run_fwd(b)
    check(b, o, lse, untouched=9.0)


@pytest.mark.parametrize("Hq,Hkv,D,page,layout", [
    (47, 1, 64, 7, "tokens"), (80, 2, 128, 1, "heads"), (160, 1, 64, 16, "tokens"), (140, 1, 128, 32, "turns"),
    (50, 1, 256, 16, "tokens")])
@pytest.mark.parametrize("lens", [[(130, 1), (17, 1), (400, 1)], [(200, 70), (33, 5), (300, 1)]], ids=["decode", "chunk"])
def test_fwd_wide_groups(lens, Hq, Hkv, D, page, layout):
    b = Batch4(lens, Hq, Hkv, D, page, layout=layout, pad_rows=1, seed=Hq)
    check(b, *run_fwd(b), untouched=9.0)


@pytest.mark.parametrize("kind", ["decode", "chunks", "mixed"])
def test_fwd_many_sequences(kind):
    n = 700
    rng = random.Random(n)
    lens = []
    for i in range(n):
        q = {"decode": 1, "chunks": rng.randint(1, 40), "mixed": 200 if i % 97 == 5 else 1}[kind]
        q = 0 if rng.random() < 0.1 else q
        lens.append((q + rng.randint(0, 60), q))
    b = Batch4(lens, 4, 2, 64, 16, seed=n)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D,group", [(64, 4), (128, 3)])
def test_fwd_one_chunk_among_single_tokens(D, group):
    lens = [(1 + 7 * i, 1) for i in range(150)]
    lens[40], lens[90], lens[91] = (700, 300), (2, 2), (40, 0)
    b = Batch4(lens, 2 * group, 2, D, 16, pad_rows=2, seed=D)
    for max_q in (300, 10 ** 6, 60):
        check(b, *run_fwd(b, max_q_len=max_q), untouched=9.0)


@pytest.mark.parametrize("lens", [[(20000, 1)], [(20000, 1), (31, 1), (9000, 3)], [(17000, 20)], [(17000, 64), (100, 1)]],
                         ids=["one", "rows", "short_chunk", "chunk"])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 64), (8, 1, 128), (4, 1, 256)])
def test_fwd_long_caches(lens, Hq, Hkv, D):
    b = Batch4(lens, Hq, Hkv, D, 16, seed=5)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D,dtype,page,layout", [(64, HF, 16, "heads"), (64, BF, 7, "tokens"), (128, BF, 64, "heads"),
                                                 (128, HF, 24, "turns"), (128, BF, 16, "tokens")])
def test_fwd_more_units_than_blocks(D, dtype, page, layout):
    """Batches whose units are shared out over teams of a block's warps: units of one tile, of many, cut by
    several teams and by several blocks, places without rows, and the same bits whatever the workspace held."""
    rng = random.Random(D + page)
    lens = [(rng.choice([1, 2, 31, 130, 700]), 1) for _ in range(330)]
    lens[7], lens[200], lens[329] = (30000, 1), (5000, 1), (9000, 1)
    lens[50] = lens[51] = (0, 0)
    b = Batch4(lens, 2, 1, D, page, dtype, layout=layout, pad_rows=2, seed=D)
    ws = torch.full((fa.attn_paged_coded_fwd_workspace_size(b.T, 1, 2, 1, D, page),), 255, dtype=torch.uint8, device="cuda")
    first = run_fwd(b, workspace=ws)
    check(b, *first, untouched=9.0)
    for _ in range(3):
        again = run_fwd(b, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    b = Batch4([(257, 1)] * 160, 8, 2, D, page, dtype, layout=layout, seed=1)
    check(b, *run_fwd(b))
    b = Batch4([(64, 3)] * 200, 4, 2, D, page, dtype, layout=layout, seed=2)  # six rows a head
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D,rows", [(64, 3), (64, 5), (64, 7), (128, 3), (128, 5), (256, 1), (256, 3)])
def test_fwd_more_units_than_blocks_of_many_rows(D, rows):
    """As above with four heads a head, so up to four blocks of rows, and head size 256."""
    rng = random.Random(D + rows)
    lens = [(rng.choice([rows, 40, 150]), rows) for _ in range(330)]
    lens[3], lens[100], lens[329] = (12000, rows), (0, 0), (3000, rows)
    b = Batch4(lens, 4, 1, D, 16, HF if rows == 3 else BF, layout="heads", pad_rows=1, seed=D)
    first = run_fwd(b)
    check(b, *first, untouched=9.0)
    again = run_fwd(b)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_fwd_one_long_sequence_among_many():
    b = Batch4([(30000, 1)] + [(x, 1) for x in range(1, 200)], 4, 1, 64, 16, seed=3)
    check(b, *run_fwd(b))
    b = Batch4([(30000, 40), (3, 3)] + [(100 + i, 50) for i in range(30)], 2, 1, 64, 16, seed=3)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", ["verify", "mixed"])
def test_fwd_every_key_visible(name, D):
    b = Batch4(VERIFY if name == "verify" else MIXED, 4, 2, D, 16, causal=0, seed=D)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("D,group", [(64, 1), (128, 4), (256, 2)])
def test_fwd_rows_without_keys_and_empty_sequences(D, group):
    lens = [(0, 1), (3, 7), (0, 0), (40, 0), (0, 130), (100, 300), (5, 1)]
    b = Batch4(lens, 2 * group, 2, D, 16, pad_rows=5, seed=2)
    check(b, *run_fwd(b), untouched=9.0)
    b = Batch4([(0, 0), (0, 0)], 2 * group, 2, D, 16, pad_rows=5, seed=2)
    check(b, *run_fwd(b), untouched=9.0)


@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
@pytest.mark.parametrize("max_q", [1, 3, 100000])
def test_fwd_is_right_for_any_max_q_len(lens, max_q):
    b = Batch4(lens, 8, 2, 128, 16, seed=4)
    o, lse = run_fwd(b, max_q_len=max_q)
    check(b, o, lse)
    o2, lse2 = run_fwd(b, max_q_len=max_q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("stale", [0x7f, 0xff, 0x7e])
@pytest.mark.parametrize("lens", [[(33, 1), (130, 1)], [(200, 150), (33, 20)]], ids=["rows", "tiles"])
@pytest.mark.parametrize("page", [64, 24])
def test_fwd_stale_rows_have_no_influence(lens, stale, page):
    b = Batch4(lens, 4, 1, 128, page, stale=stale, seed=1)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "n_pages"])
@pytest.mark.parametrize("lens", [[(100, 1), (300, 1)], [(100, 40), (300, 200)]], ids=["rows", "tiles"])
@pytest.mark.parametrize("page", [16, 32, 100, 7])
def test_fwd_entries_that_name_no_page(lens, bad, page):
    b = Batch4(lens, 4, 2, 64, page, seed=7)
    where = [(0, 0), (1, 1), (1, 2)]
    for s, col in where:
        b.table[s, col] = b.n_pages if bad == "n_pages" else bad
    check(b, *run_fwd(b), bad_pages=where)


def test_fwd_no_page_at_all():
    b = Batch4([(100, 1), (300, 150)], 4, 2, 64, 16, seed=7)
    b.table[:] = -1
    o, lse = run_fwd(b)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_fwd_lengths_that_are_out_of_range():
    b = Batch4([(64, 2), (64, 3)], 4, 2, 64, 16, extra_cols=0, seed=9)
    a = b.on_gpu()
    want, _, tol, _ = b.reference()
    a["kv_lens"] = torch.tensor([2 ** 31 - 1, -9], dtype=I32, device="cuda")
    a["cu_q"] = torch.tensor([-5, 2, 2 ** 31 - 1], dtype=I32, device="cuda")
    for max_q in (1, 1000):
        o, lse = fa.attn_paged_coded_fwd(**a, max_q_len=max_q, causal=1, scale=b.scale)
        ok()
        assert (np.abs(o.double().cpu().numpy() - want)[:2] <= tol[:2]).all()
        assert (o[2:] == 0).all() and torch.isneginf(lse[:, 2:]).all()
    a["cu_q"] = torch.tensor([4, 1, 0], dtype=I32, device="cuda")  # falling: no rows
    o = torch.full_like(a["q"], 9.0)
    fa.attn_paged_coded_fwd(**a, max_q_len=1, o=o)
    ok()
    assert (o == 9.0).all()


@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_fwd_units_and_sharp_logits(lens, D):
    b = Batch4(lens, 4, 2, D, 16, k_unit=0.037, v_unit=13.0, seed=11, q_sigma=8.0)
    check(b, *run_fwd(b))


@pytest.mark.parametrize("exponent", [-120, -40, 30, 100])
@pytest.mark.parametrize("lens", [DECODE, MIXED], ids=["decode", "mixed"])
def test_fwd_queries_far_from_fp16(lens, exponent):
    """bf16 queries that fp16 does not hold: rows near the ends of bf16's range, and elements of one row that
    lie far apart."""
    b = Batch4(lens, 4, 2, 128, 16, seed=17)
    b.q = b.q * torch.where(torch.arange(128) % 3 == 0, 1.0, 2.0 ** -12).to(BF) * 2.0 ** exponent
    b.scale = b.scale * 2.0 ** -exponent if exponent < 100 else 2.0 ** -exponent
    check(b, *run_fwd(b))


@pytest.mark.parametrize("max_q", [1, 1000])
def test_fwd_infinite_and_nan_queries_stay_in_their_rows(max_q):
    b = Batch4([(50, 2), (60, 1)], 4, 2, 128, 16, seed=12)
    o, lse = run_fwd(b, max_q_len=max_q)
    check(b, o, lse)
    b.q[0, 1, 7], b.q[2, 3, 9] = float("nan"), float("inf")
    o2, lse2 = run_fwd(b, max_q_len=max_q)
    assert torch.isnan(o2[0, 1].float()).all() and torch.isnan(lse2[1, 0])
    assert not torch.isfinite(o2[2, 3].float()).any()
    for t in range(3):
        for h in range(4):
            if (t, h) not in ((0, 1), (2, 3)):
                assert torch.equal(o[t, h], o2[t, h]) and lse[h, t] == lse2[h, t]
    b = Batch4([(50, 1), (60, 1)], 4, 2, 128, 64, seed=12)
    b.k_scales[int(b.table[0, 0]), 3] = 0x7f  # a seen key of the first sequence
    o, lse = run_fwd(b, max_q_len=max_q)
    assert torch.isnan(o[0].float()).all() and torch.isnan(lse[:, 0]).all() and torch.isfinite(o[1].float()).all()


@pytest.mark.parametrize("D", [64, 128])
def test_fwd_wide_rows_of_a_fused_projection(D):
    b = Batch4(MIXED, 8, 2, D, 16, seed=6)
    a = b.on_gpu()
    x = torch.randn(b.T, 12, D, device="cuda").to(BF)
    x[:, :8] = a["q"]
    a["q"] = x[:, :8]
    wide = torch.full((len(b.lens), b.table.shape[1] + 5), 2 ** 30, dtype=I32, device="cuda")
    wide[:, :b.table.shape[1]] = a["block_table"]
    a["block_table"] = wide[:, :b.table.shape[1]]
    a["k_scales"], a["v_scales"] = (a[x].view(torch.float8_e4m3fn) for x in ("k_scales", "v_scales"))
    for max_q in (1, None):
        check(b, *fa.attn_paged_coded_fwd(**a, max_q_len=max_q, scale=b.scale))
        ok()
    o, none = fa.attn_paged_coded_fwd(**a, want_lse=False)
    assert none is None


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_past_32_bits(D):
    """A cache of more than 2^32 bytes of codes whose used pages are the last ones."""
    page, Hkv = 64, 8
    first = (9 << 29) // (page * Hkv * D // 2)
    b = Batch4([(200, 1), (513, 70)], 16, Hkv, D, page, first_page=first, seed=8)
    assert b.k_codes.numel() > 1 << 32
    for max_q in (1, 70):
        check(b, *run_fwd(b, max_q_len=max_q))
    rows = torch.randn(2, Hkv, D, device="cuda").to(BF)
    slots = torch.tensor([b.n_pages * page - 1, 5], device="cuda")
    fa.attn_paged_coded_append(rows, rows, slots, b.k_codes, b.k_scales, b.v_codes, b.v_scales)
    ok()
    c, s = encode(rows.float().cpu().numpy(), 1.0)
    for codes, scales in ((b.k_codes, b.k_scales), (b.v_codes, b.v_scales)):
        assert np.array_equal(codes[-1, -1].cpu().numpy(), c[0]) and np.array_equal(codes[0, 5].cpu().numpy(), c[1])
        assert np.array_equal(scales[-1, -1].cpu().numpy(), s[0]) and np.array_equal(scales[0, 5].cpu().numpy(), s[1])


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_fwd_writes_inside_its_buffers(lens, D):
    b = Batch4(lens, 8, 2, D, 16, seed=13)
    a = b.on_gpu()
    max_q = max(n for _, n in lens)
    o, lse = Guarded((b.T, 8, D), BF), Guarded((8, b.T), torch.float32)
    size = fa.attn_paged_coded_fwd_workspace_size(b.T, max_q, 8, 2, D, 16)
    ws = Guarded((max(size, 4),), torch.uint8)
    fa.attn_paged_coded_fwd(**a, max_q_len=max_q, scale=b.scale, o=o.t, lse=lse.t, workspace=ws.t)
    ok()
    assert o.guards_intact() and lse.guards_intact() and ws.guards_intact()
    assert o.fully_written() and lse.fully_written()
    check(b, o.t, lse.t)


@pytest.mark.parametrize("lens,max_q", [([(20000, 1), (9000, 1), (40, 1)], 1), ([(20000, 100), (300, 1), (8000, 1)], 100)],
                         ids=["rows", "mixed"])
def test_fwd_workspace_contents_do_not_matter(lens, max_q):
    b = Batch4(lens, 8, 1, 128, 16, seed=30)
    size = fa.attn_paged_coded_fwd_workspace_size(b.T, max_q, 8, 1, 128, 16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = None
    g = torch.Generator(device="cuda").manual_seed(1)
    for fill in ("zero", "ones", "random", "as left", "as left"):
        if fill == "ones":
            ws.fill_(255)
        elif fill == "random":
            ws.copy_(torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda", generator=g))
        o, lse = run_fwd(b, max_q_len=max_q, workspace=ws)
        if first is None:
            first = (o, lse)
            check(b, o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), fill


def test_two_graphs_that_share_a_workspace():
    bs = [Batch4([(20000, 1), (37, 1)], 8, 1, 128, 16, seed=31), Batch4([(9000, 60), (500, 1)], 8, 1, 128, 16, seed=32)]
    size = max(fa.attn_paged_coded_fwd_workspace_size(b.T, 60, 8, 1, 128, 16) for b in bs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for b, max_q in zip(bs, (1, 60)):
        a = b.on_gpu()
        o = torch.empty_like(a["q"])
        lse = torch.empty((8, b.q.shape[0]), dtype=torch.float32, device="cuda")
        args = dict(a, max_q_len=max_q, scale=b.scale, o=o, lse=lse, workspace=ws)
        fa.attn_paged_coded_fwd(**args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.attn_paged_coded_fwd(**args)
        graphs.append((g, a))
        outs.append((o, lse))
    for i in (0, 0, 1, 0, 1, 1, 0):
        outs[i][0].fill_(9.0)
        graphs[i][0].replay()
    ok()
    for b, (o, lse) in zip(bs, outs):
        check(b, o, lse)


@pytest.mark.parametrize("kind", ["zero", "stream", "handle"])
def test_streams_in_every_form(kind):
    side = torch.cuda.Stream()
    stream = {"zero": 0, "stream": side, "handle": side.cuda_stream}[kind]
    b = Batch4([(9000, 1), (40, 1)], 8, 1, 64, 16, seed=40)
    a = b.on_gpu()
    torch.cuda.synchronize()
    for _ in range(3):
        o, lse = fa.attn_paged_coded_fwd(**a, max_q_len=1, scale=b.scale, stream=stream)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # on the current stream
        del junk
    k = torch.randn(1, 1, 64, device="cuda").to(BF)
    slot = torch.tensor([int(b.table[1, 2]) * 16 + 8], device="cuda")
    torch.cuda.synchronize()
    fa.attn_paged_coded_append(k, k, slot, b.k_codes, b.k_scales, b.v_codes, b.v_scales, stream=stream)
    torch.cuda.synchronize()
    ok()
    check(b, o, lse)
    assert np.array_equal(b.k_codes[int(b.table[1, 2]), 8].cpu().numpy(), encode(k[0].float().cpu().numpy(), 1.0)[0])


def test_refusals_launch_nothing():
    b = Batch4([(4000, 1)], 8, 2, 128, 16, seed=1)
    a = b.on_gpu()
    size = fa.attn_paged_coded_fwd_workspace_size(b.T, 1, 8, 2, 128, 16)
    before = fa.attn_kernel_launches()
    k = torch.zeros(1, 2, 128, dtype=BF, device="cuda")
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    cache = [a[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    for over in (dict(workspace=torch.empty(size - 256, dtype=torch.uint8, device="cuda")), dict(q=a["q"].float()),
                 dict(cu_q=a["cu_q"].long()), dict(kv_lens=a["kv_lens"].repeat(2)), dict(block_table=a["block_table"].t()),
                 dict(v_codes=a["v_codes"][:, :8]), dict(q=a["q"][:, :7]), dict(k_scales=a["k_scales"][..., :4]),
                 dict(k_codes=a["k_codes"].view(torch.int8)), dict(o=torch.empty(1, 8, 128, device="cuda")),
                 dict(lse=torch.empty(1, 8, device="cuda")), dict(kv_lens=a["kv_lens"].cpu()), dict(k_unit=0.0),
                 dict(v_unit=float("inf")), dict(k_unit=1e-45), dict(scale=1e-30, k_unit=1e-30)):
        with pytest.raises(fa.AttnError):
            fa.attn_paged_coded_fwd(**{**a, "max_q_len": 1, **over})
    for bad in ([k.float(), k.float(), slot, *cache], [k, k[:, :1], slot, *cache], [k, k, slot.int(), *cache],
                [k, k, slot, cache[0], cache[1], cache[0], cache[3]], [k[..., :64], k[..., :64], slot, *cache]):
        with pytest.raises(fa.AttnError):
            fa.attn_paged_coded_append(*bad)
    assert fa.attn_kernel_launches() == before


# ------------------------------------------------------------------ a run of them
class Server4:
    """A cache in 4 bits of growing, forking and ending sequences; the host keeps a dense copy."""

    def __init__(self, n, Hq, Hkv, D, page, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.Hq, self.Hkv, self.D, self.page, self.n_pages = n, Hq, Hkv, D, page, 200
        self.codes, self.scales = place((self.n_pages, page, Hkv, D // 2), "heads", 0x77), place((self.n_pages, page, Hkv, D // 16), "heads", 0x7f)
        i32 = dict(dtype=I32, device="cuda")
        self.table = torch.full((n, 40), -1, **i32)
        self.free = torch.randperm(self.n_pages, generator=self.g, **i32)
        self.head, self.ctx, self.shares = torch.zeros(1, **i32), torch.zeros(n, **i32), torch.zeros(self.n_pages, **i32)
        self.dense = [[np.zeros((0, Hkv, D))] * 2 for _ in range(n)]

    def tokens(self, new):
        cap = sum(new) + 3
        x = torch.randn(cap, self.Hq + 2 * self.Hkv, self.D, device="cuda", generator=self.g).to(BF)
        q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
        cu, kv, slots, counts = fa.attn_paged_tables(self.ctx, torch.tensor(new, dtype=I32, device="cuda"), self.free, self.table,
                                                     self.page, cap, free_head=self.head)
        cache = (self.codes[0], self.scales[0], self.codes[1], self.scales[1])
        fa.attn_paged_coded_append(k, v, slots, *cache)
        o, lse = fa.attn_paged_coded_fwd(q, *cache, self.table, cu, kv, max_q_len=max(new))
        self.ctx.copy_(kv)
        self.head.copy_(counts[1:2])
        ok()
        assert counts.tolist()[2:] == [0, 0]
        at = 0
        for s, m in enumerate(new):
            if m == 0:
                continue
            self.dense[s] = [np.concatenate([d, decode(*encode(y[at:at + m].float().cpu().numpy(), 1.0), 1.0)])
                             for d, y in zip(self.dense[s], (k, v))]
            b = Batch4([(self.dense[s][0].shape[0], m)], self.Hq, self.Hkv, self.D, self.page)
            b.q, b.dense, b.scale = q[at:at + m].cpu(), [tuple(self.dense[s])], self.D ** -0.5
            check(b, o[at:at + m], lse[:, at:at + m])
            at += m

    def fork(self, parents, lens=None):
        copies, counts = fa.attn_paged_fork(torch.tensor(parents, dtype=I32, device="cuda"), self.ctx, self.free, self.table,
                                            self.page, self.shares, free_head=self.head,
                                            lens=None if lens is None else torch.tensor(lens, dtype=I32, device="cuda"))
        fa.attn_paged_copy(copies, [*self.codes, *self.scales])
        self.head.copy_(counts[1:2])
        for i, p in enumerate(parents):
            if p >= 0:
                self.dense[i] = [d[:self.dense[p][0].shape[0] if lens is None else lens[i]] for d in self.dense[p]]
        ok()

    def cut(self, keep):
        keep = torch.tensor(keep, dtype=I32, device="cuda")
        counts = fa.attn_paged_free(self.ctx, keep, self.table, self.page, self.shares, self.free, self.head)
        self.ctx.copy_(torch.minimum(self.ctx, keep))
        self.head.copy_(counts[1:2])
        self.dense = [[d[:m] for d in x] for x, m in zip(self.dense, self.ctx.tolist())]
        ok()
        return counts.tolist()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 24)])
def test_a_server_that_forks_and_frees(D, page):
    sv = Server4(6, 4, 2, D, page, seed=D)
    sv.tokens([100, 7, 0, 0, 0, 0])
    sv.fork([-1, -1, 0, 0, 1, -1])                     # rows 2 and 3 go on from row 0, row 4 from row 1
    for new in ([1, 1, 1, 1, 1, 0], [5, 5, 5, 5, 5, 0]):
        sv.tokens(new)
    big = 10 ** 6
    assert sv.cut([big, big, 103, big, 0, big])[2:] == [0, 0]   # row 2 loses drafted tokens, row 4 ends
    sv.fork([-1, -1, -1, -1, 3, 0], lens=[0, 0, 0, 0, 70, 96])
    sv.tokens([1, 1, 1, 1, 130, 3])
    sv.cut([0, big, big, big, big, big])                        # the first prompt's own row ends, its pages live on
    sv.tokens([33, 1, 1, 2, 1, 1])
    assert sv.cut([0] * 6)[2:] == [0, 0]
    assert int(sv.head) == 0 and sorted(sv.free.tolist()) == list(range(sv.n_pages)) and (sv.shares == 0).all()


def test_format_is_exact_in_fp16():
    """Every code times every finite scale is a number of fp16."""
    products = np.multiply.outer(E2M1, E4M3[:127]).ravel()
    assert (products.astype(np.float16).astype(np.float64) == products).all()
