"""Cases that measure the paged cache in 4 bits and the bookkeeping of shared pages of libattn: the write
of new keys and values in 4 bits, attention over them, and forking, freeing and copying pages.

`own = False` computes the operators in plain torch; `own = True` calls libattn.

A cache in 4 bits holds an element as code x block scale x unit: codes are e2m1 (two to a byte, the first
in the low half), one e4m3 scale stands for 16 elements of a head's row, the unit is a number for the
whole cache.  Codes are compared bit by bit: the format's definition leaves none of them open.
"""
import math
import random

import torch

own = False

F32 = torch.float32
I64 = torch.int64
E4M3 = torch.float8_e4m3fn
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the codes 0 to 7; 8 to 15 are their negatives


# ------------------------------------------------------------------ cases
def listed():
    """What each stands for in real use is said above it."""
    return [
        # one step of a beam search: every beam goes on from one of its prompt's beams, in rows that were empty
        _case("fork_beams_128", op="fork", n_seqs=128, n_forks=64, page=16, ctx_lo=100, ctx_hi=8000),
        # many new requests that begin with a part of the prompts of a few
        _case("fork_prefix_1024", op="fork", n_seqs=1024, n_forks=900, n_parents=32, page=64, ctx_lo=500, ctx_hi=16000,
              part=True),
        # drafted tokens that were not accepted, given back by every request of a step
        _case("free_drafts_256", op="free", n_seqs=256, page=16, ctx_lo=100, ctx_hi=4000, drop=8, n_pages=70000),
        # requests that end, half of them with a shared beginning
        _case("free_ended_1024", op="free", n_seqs=1024, page=64, ctx_lo=0, ctx_hi=30000, drop=0, shared=40,
              n_pages=270000),
        # the partly filled pages of a few forks, in one layer's cache of 16 bits
        _case("copy_8x2", op="copy", n_copies=8, pad=56, n_caches=2, Hkv=8, D=128, page=16, n_pages=300),
        # the same for all layers of a model at once: 32 of them, pages of 64, stored head by head in 4 bits
        _case("copy_64x64_e2m1", op="copy", n_copies=64, pad=64, n_caches=64, Hkv=8, D=128, page=64, n_pages=400,
              four=True, heads_first=True),
        # one decode step's cache write: 64 single tokens cut out of a fused projection
        _case("append_decode_64", op="append", tokens=64, Hq=32, Hkv=8, D=128, page=16, n_pages=4096, fused=True),
        # the prompts of many requests at once, padded to a fixed count
        _case("append_prompts_65000", op="append", tokens=65000, Hkv=16, D=64, page=128, n_pages=600, f16=True, pad=536,
              heads_first=True),
        # one user, one token, a short context: latency
        _case("decode_1x1000", op="fwd", n_seqs=1, Hq=32, Hkv=8, ctx_lo=1000, ctx_hi=1000, page=16),
        # a decode batch of unlike lengths, captured for 160 requests of which 144 are there
        _case("decode_ragged_144", op="fwd", n_seqs=160, n_empty=16, Hq=64, Hkv=8, ctx_lo=300, ctx_hi=8000, page=64,
              pad=16, heads_first=True),
        # drafted tokens being verified: five new tokens a request
        _case("verify_16x5", op="fwd", n_seqs=16, n_chunks=16, q_lo=5, q_hi=5, Hq=32, Hkv=8, D=64, ctx_lo=2000,
              ctx_hi=6000, page=32, f16=True),
        # the benchmark's chunked prefill over a cache in 4 bits
        _case("chunk_512x32768", op="fwd", n_seqs=1, n_chunks=1, q_lo=512, q_hi=512, Hq=64, Hkv=8, ctx_lo=32256,
              ctx_hi=32256, page=64, heads_first=True),
    ]


def _case(name, **kw):
    base = dict(name=name, op="fwd", n_seqs=1, n_chunks=0, n_empty=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0, Hq=32, Hkv=8,
                D=128, page=16, causal=1, f16=False, pad=0, heads_first=False, fused=False, tokens=0, n_pages=0,
                n_forks=0, n_parents=0, part=False, drop=0, shared=0, n_copies=0, n_caches=2, four=False,
                k_unit=1.0, v_unit=1.0)
    base.update(kw)
    return base


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the same ranges."""
    what = rng.choice(["fork", "free", "copy", "append", "append", "decode", "decode", "verify", "mixed", "chunk", "prefill"])
    f16 = rng.random() < 0.4
    page = rng.choice([16, 16, 24, 32, 48, 64, 128, 256])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    heads_first = rng.random() < 0.5
    if what == "fork":
        n = _log(rng, 2, 1024)
        forks = rng.randint(1, n - 1)
        return _case("", op="fork", n_seqs=n, n_forks=forks, n_parents=rng.randint(1, n - forks), page=page,
                     ctx_lo=1, ctx_hi=_log(rng, 100, 16000), part=rng.random() < 0.5)
    if what == "free":
        n, hi = _log(rng, 1, 1024), _log(rng, 100, 16000)
        shared = rng.choice([0, 20, 100])
        return _case("", op="free", n_seqs=n, page=page, ctx_lo=0, ctx_hi=hi, drop=rng.choice([0, 1, 9, 200]),
                     shared=shared, n_pages=n * _ceil(hi, page) + rng.randint(100, 1000))
    if what == "copy":
        n, row = _log(rng, 1, 64), page * Hkv * D * 2
        caches = min(64, 2 * max(1, _log(rng, 1, 32)), max(2, 2 * int(250_000_000 // (n * row) // 2)))
        return _case("", op="copy", n_copies=n, pad=rng.randint(0, 64), n_caches=caches, Hkv=Hkv, D=D, page=page,
                     n_pages=2 * n + rng.randint(1, 40), four=rng.random() < 0.5, heads_first=heads_first)
    unit = rng.choice([1.0, 1.0, 0.5, 0.04])
    if what == "append":
        t = _log(rng, 1, 65000 if D * Hkv <= 1024 else 20000)
        return _case("", op="append", tokens=t, Hq=2 * Hkv, Hkv=Hkv, D=D, page=page, n_pages=t // page + rng.randint(2, 90),
                     f16=f16, pad=rng.randint(0, 60), fused=rng.random() < 0.5, heads_first=heads_first, k_unit=unit)
    kw = dict(op="fwd", Hq=Hkv * group, Hkv=Hkv, D=D, page=page, f16=f16, heads_first=heads_first, k_unit=unit,
              v_unit=rng.choice([1.0, 0.3]))
    if what == "decode":
        n = _log(rng, 1, 128)
        hi = _log(rng, 64, min(60000, 2_000_000 // (n * Hkv)))
        return _case("", n_seqs=n + 3, n_empty=3, ctx_lo=hi // 8, ctx_hi=hi, pad=rng.randint(0, 20), **kw)
    if what == "verify":
        n = _log(rng, 1, 64)
        hi = _log(rng, 64, min(30000, 1_000_000 // (n * Hkv)))
        return _case("", n_seqs=n, n_chunks=n, q_lo=2, q_hi=rng.randint(2, 9), ctx_lo=hi // 4, ctx_hi=hi, **kw)
    if what == "mixed":
        q, hi = rng.randint(16, 700), _log(rng, 100, 6000)
        n = max(4, min(rng.randint(4, 40), 1_000_000_000 // (kw["Hq"] * q * (hi + q))))
        return _case("", n_seqs=n, n_chunks=rng.randint(1, 4), q_lo=10, q_hi=q, ctx_lo=0, ctx_hi=hi,
                     pad=rng.randint(0, 9), **kw)
    if what == "chunk":
        q = _log(rng, 16, 1024)
        return _case("", n_seqs=1, n_chunks=1, q_lo=q, q_hi=q, ctx_lo=0, ctx_hi=_log(rng, 100, 16000), **kw)
    n = rng.randint(1, 4)
    hi = _log(rng, 100, min(4000, int(math.sqrt(1_000_000_000 // (n * kw["Hq"])))))
    return _case("", n_seqs=n, n_chunks=n, q_lo=1, q_hi=hi, causal=rng.randint(0, 1), **kw)


def _ceil(a, b):
    return -(-a // b)


def _rng(case):
    return random.Random("%(n_seqs)d %(n_forks)d %(q_hi)d %(ctx_lo)d %(ctx_hi)d %(drop)d %(page)d" % case)


def _lens(case):
    """Cached and new tokens of every sequence of an attention case: lists that depend on the case alone."""
    r = _rng(case)
    n = case["n_seqs"]
    q = [r.randint(case["q_lo"], case["q_hi"]) if i < case["n_chunks"] else 1 for i in range(n)]
    q = [0 if i >= n - case["n_empty"] else x for i, x in enumerate(q)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    both = [(c, x) if x else (0, 0) for c, x in zip(ctx, q)]
    live = both[:n - case["n_empty"]]
    r.shuffle(live)
    both[:len(live)] = live
    return [b[0] for b in both], [b[1] for b in both]


def _fork_plan(case):
    """(tokens, parents, tokens that a fork takes) of every row; rows without tokens are what forks go to."""
    r = _rng(case)
    n, forks = case["n_seqs"], case["n_forks"]
    live = n - forks
    kv = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(live)] + [0] * forks
    sources = r.sample(range(live), min(case["n_parents"] or live, live))
    parents = [-1] * live + [r.choice(sources) for _ in range(forks)]
    take = [0] * live + [r.randint(1, kv[p]) if case["part"] else kv[p] for p in parents[live:]]
    order = list(range(n))
    r.shuffle(order)  # row order[i] is what row i was
    at = [0] * n
    for i, x in enumerate(order):
        at[x] = i
    return [kv[x] for x in order], [at[parents[x]] if parents[x] >= 0 else -1 for x in order], [take[x] for x in order]


def _free_plan(case):
    """(tokens, tokens that are kept, pages at the front that are shared) of every row; drop 0: the row ends."""
    r = _rng(case)
    kv = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["n_seqs"])]
    keep = [max(0, x - r.randint(0, case["drop"])) if case["drop"] else 0 for x in kv]
    front = [min(case["shared"], x // case["page"]) if r.random() < 0.5 else 0 for x in kv]
    return kv, keep, front


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _place(shape, dtype, heads_first):
    """An empty cache [n_pages, page, heads, x], stored token by token or head by head."""
    n, page, H, x = shape
    if heads_first:
        return torch.empty((n, H, page, x), dtype=dtype, device="cuda").transpose(1, 2)
    return torch.empty(shape, dtype=dtype, device="cuda")


def _cache4(case, n_pages, g):
    """(codes, scales) of normal values."""
    page, H, D = case["page"], case["Hkv"], case["D"]
    codes = _place((n_pages, page, H, D // 2), torch.uint8, case["heads_first"])
    scales = _place((n_pages, page, H, D // 16), E4M3, case["heads_first"])
    step = max(1, (1 << 24) // (page * H * D))
    for a in range(0, n_pages, step):
        b = min(a + step, n_pages)
        codes[a:b], scales[a:b] = _encode(_normal((b - a, page, H, D), F32, g))
    return codes, scales


def _table(pages, counts, width):
    """A block table whose row i holds the next counts[i] of `pages`, and -1 behind them."""
    c = torch.tensor(counts, device="cuda")
    cols = torch.arange(width, device="cuda")
    first = torch.cumsum(c, 0) - c
    at = (first[:, None] + cols).clamp(max=max(len(pages) - 1, 0))
    filled = cols < c[:, None]
    if len(pages) == 0:
        return torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    return torch.where(filled, pages[at], torch.full_like(pages[at], -1))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    return {"fork": _prepare_fork, "free": _prepare_free, "copy": _prepare_copy, "append": _prepare_append,
            "fwd": _prepare_fwd}[case["op"]](case, s, g)


def _prepare_fork(case, s, g):
    kv, parents, take = _fork_plan(case)
    page = case["page"]
    have = [_ceil(x, page) for x in kv]
    spare = case["n_forks"] + 20
    n_pages = sum(have) + spare
    pages = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    s["block_table"] = _table(pages[spare:], have, max(max(have), 1) + 2)
    s["free_pages"] = pages[:spare].contiguous()
    s["shares"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    s["kv_lens"], s["parents"] = _ints(kv), _ints(parents)
    s["lens"] = _ints(take) if case["part"] else None
    return s


def _prepare_free(case, s, g):
    kv, keep, front = _free_plan(case)
    page, n_pages = case["page"], case["n_pages"]
    have = [_ceil(x, page) for x in kv]
    pages = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    used = sum(have)
    table = _table(pages[:used], have, max(max(have), 1) + 2)
    shares = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    rows = torch.tensor([i for i, x in enumerate(front) if x], dtype=I64, device="cuda")
    if len(rows):  # rows with a shared front take the columns of the first row that has them all
        full = max(range(len(front)), key=lambda i: front[i])
        cols = torch.arange(table.shape[1], device="cuda")
        n_front = _ints(front)[rows]
        theirs = cols < n_front[:, None]
        table[rows] = torch.where(theirs, table[full], table[rows])
        of = torch.where(theirs, table[full].expand(len(rows), -1), n_pages).reshape(-1).long()
        names = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
        names.index_add_(0, of, torch.ones_like(of, dtype=torch.int32))
        shares = (names[:n_pages] - 1).clamp(min=0)
    s["block_table"], s["shares"] = table, shares
    s["kv_lens"], s["keep_lens"] = _ints(kv), _ints(keep)
    s["free_pages"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    s["free_pages"][used:] = pages[used:]
    s["free_head"] = _ints([used])
    return s


def _prepare_copy(case, s, g):
    n, page, H, D, m = case["n_copies"], case["page"], case["Hkv"], case["D"], case["n_caches"]
    n_pages = case["n_pages"]
    pages = torch.randperm(n_pages - 1, device="cuda", generator=g, dtype=torch.int32)  # the last page is nobody's
    copies = torch.full((n + case["pad"], 3), -1, dtype=torch.int32, device="cuda")
    src = pages[torch.randint(n_pages - 1 - n, (n,), device="cuda", generator=g)]
    rows = torch.randint(1, page + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    at = torch.randperm(n + case["pad"], device="cuda", generator=g)[:n]
    copies[at] = torch.stack([src, pages[n_pages - 1 - n:], rows], 1)
    s["copies"] = copies
    shape = (m, n_pages, H, page) if case["heads_first"] else (m, n_pages, page, H)
    if case["four"]:
        s["all"] = [torch.randint(256, (*shape, x), dtype=torch.uint8, device="cuda", generator=g) for x in (D // 2, D // 16)]
    else:
        s["all"] = [_normal((*shape, D), torch.bfloat16, g)]
    if case["heads_first"]:
        s["all"] = [x.transpose(2, 3) for x in s["all"]]
    s["caches"] = [c for x in s["all"] for c in x]
    return s


def _prepare_append(case, s, g):
    dtype = torch.float16 if case["f16"] else torch.bfloat16
    T, n_pages, page, Hq, Hkv, D = (case[x] for x in ("tokens", "n_pages", "page", "Hq", "Hkv", "D"))
    rows = T + case["pad"]
    if case["fused"]:  # q, k and v of one projection
        x = _normal((rows, Hq + 2 * Hkv, D), dtype, g)
        s["k"], s["v"] = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        s["k"], s["v"] = _normal((rows, Hkv, D), dtype, g), _normal((rows, Hkv, D), dtype, g)
    slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:rows]
    slots[T:] = -1  # the rows that pad the batch
    s["slot_map"] = slots
    for name in ("k", "v"):
        for x, dt, n in (("codes", torch.uint8, D // 2), ("scales", E4M3, D // 16)):
            s[name + "_" + x] = _place((n_pages, page, Hkv, n), dt, case["heads_first"])
            s[name + "_" + x].view(torch.uint8).zero_()
    return s


def _prepare_fwd(case, s, g):
    dtype = torch.float16 if case["f16"] else torch.bfloat16
    page, Hq, Hkv, D = case["page"], case["Hq"], case["Hkv"], case["D"]
    ctx, new = _lens(case)
    s["ctx"], s["new"] = ctx, new
    want = [_ceil(c + x, page) for c, x in zip(ctx, new)]
    n_pages = sum(want) + 7
    pages = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    s["block_table"] = _table(pages, want, max(want) + 3)
    s["k_codes"], s["k_scales"] = _cache4(case, n_pages, g)
    s["v_codes"], s["v_scales"] = _cache4(case, n_pages, g)
    T = sum(new) + case["pad"]
    s["q"] = _normal((T, Hq, D), dtype, g)
    s["scale"] = 1.0 / (math.sqrt(D) * case["k_unit"])  # logits of the same spread for any unit
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu_q"], s["kv_lens"] = _ints(cu), _ints([c + x for c, x in zip(ctx, new)])
    s["cu"], s["max_q_len"], s["max_kv"] = cu, max(new), max(c + x for c, x in zip(ctx, new))
    s["o"] = torch.zeros((T, Hq, D), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((Hq, T), dtype=F32, device="cuda")
    if own:
        import attention_forward_11_gb300 as fa
        size = fa.attn_paged_coded_fwd_workspace_size(T, s["max_q_len"], Hq, Hkv, D, page)
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import attention_forward_11_gb300 as fa
        if op == "fork":
            copies, counts = fa.attn_paged_fork(s["parents"], s["kv_lens"], s["free_pages"], s["block_table"], case["page"],
                                                s["shares"], lens=s["lens"])
            return s["block_table"], s["kv_lens"], s["shares"], copies, counts
        if op == "free":
            counts = fa.attn_paged_free(s["kv_lens"], s["keep_lens"], s["block_table"], case["page"], s["shares"],
                                        s["free_pages"], s["free_head"])
            return s["shares"], s["free_pages"], counts
        if op == "copy":
            fa.attn_paged_copy(s["copies"], s["caches"])
            return s["all"]
        if op == "append":
            fa.attn_paged_coded_append(s["k"], s["v"], s["slot_map"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                  k_unit=case["k_unit"], v_unit=case["v_unit"])
            return s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]
        return fa.attn_paged_coded_fwd(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["block_table"],
                                  s["cu_q"], s["kv_lens"], max_q_len=s["max_q_len"], causal=case["causal"],
                                  scale=s["scale"], k_unit=case["k_unit"], v_unit=case["v_unit"], o=s["o"], lse=s["lse"],
                                  workspace=s["workspace"])
    return {"fork": _plain_fork, "free": _plain_free, "copy": _plain_copy, "append": _plain_append, "fwd": _plain_fwd}[op](s)


def _plain_fork(s):
    page, table, kv, free, shares = s["case"]["page"], s["block_table"], s["kv_lens"], s["free_pages"], s["shares"]
    n, width = table.shape
    n_pages, n_free = len(shares), len(free)
    row = torch.arange(n, device="cuda")
    parent = s["parents"].long()
    wants = (parent >= 0) & (parent < n) & (parent != row)
    p = torch.where(wants, parent, row)
    forks = wants & ~wants[p]  # not from a row that is rewritten itself
    length = kv[p].long().clamp(0, width * page)
    if s["lens"] is not None:
        length = torch.minimum(length, s["lens"].long().clamp(min=0))
    full, rest = length // page, length % page
    theirs = table[p]
    src = theirs.gather(1, full.clamp(max=width - 1)[:, None])[:, 0].long()
    needs = forks & (rest > 0) & (src >= 0) & (src < n_pages)
    at = torch.cumsum(needs, 0) - needs.long()
    gets = needs & (at < n_free)
    dst = torch.where(gets, free[at.clamp(max=n_free - 1)].long(), -1)
    cols = torch.arange(width, device="cuda")
    shared = forks[:, None] & (cols < full[:, None])
    last = (forks & (rest > 0))[:, None] & (cols == full[:, None])
    table.copy_(torch.where(shared, theirs, torch.where(last, torch.where(needs, dst, src)[:, None].int(), table)))
    kv.copy_(torch.where(forks, length.int(), kv))
    counted = shared & (theirs >= 0) & (theirs < n_pages)
    more = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    of = torch.where(counted, theirs, n_pages).reshape(-1).long()
    more.index_add_(0, of, torch.ones_like(of, dtype=torch.int32))
    shares += more[:n_pages]
    copies = torch.where(gets[:, None], torch.stack([src, dst, rest], 1), torch.tensor([-1, -1, 0], device="cuda"))
    counts = torch.stack([forks.sum(), gets.sum(), (needs & ~gets).sum(), (wants & ~forks).sum()])
    return table, kv, shares, copies.int(), counts.int()


def _plain_free(s):
    page, table, shares, free = s["case"]["page"], s["block_table"], s["shares"], s["free_pages"]
    width = table.shape[1]
    n_pages, n_free = len(shares), len(free)
    kv, keep = s["kv_lens"].long().clamp(0, width * page), s["keep_lens"].long().clamp(min=0)
    cols = torch.arange(width, device="cuda")
    kept, had = (keep + page - 1) // page, (kv + page - 1) // page
    gone = (cols >= kept[:, None]) & (cols < had[:, None]) & (table >= 0) & (table < n_pages)
    of = torch.where(gone, table, n_pages).reshape(-1).long()
    less = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    less.index_add_(0, of, torch.ones_like(of, dtype=torch.int32))
    shares -= less[:n_pages]
    over = shares < 0
    shares.clamp_(min=0)
    last = table.gather(1, (keep // page).clamp(max=width - 1)[:, None])[:, 0].long()
    cut = (keep < kv) & (keep % page > 0) & (last >= 0) & (last < n_pages) & (shares[last.clamp(0, n_pages - 1)] > 0)
    freed = over.sum()
    head = s["free_head"].long().clamp(0, n_free)[0]
    fit = torch.minimum(freed, head)
    at = head - freed + torch.cumsum(over, 0) - 1
    to = torch.where(over & (at >= 0), at, n_free)
    room = torch.cat([free, free.new_zeros(1)])
    room.scatter_(0, to, torch.arange(n_pages, device="cuda", dtype=torch.int32))
    free.copy_(room[:n_free])
    return shares, free, torch.stack([fit, head - fit, freed - fit, cut.sum()]).int()


def _plain_copy(s):
    n_pages = s["case"]["n_pages"]
    src, dst, rows = (x.long() for x in s["copies"].unbind(1))
    there = (src >= 0) & (dst >= 0) & (rows > 0)
    src, dst, rows = torch.where(there, src, n_pages - 1), torch.where(there, dst, n_pages - 1), torch.where(there, rows, 0)
    mine = (torch.arange(s["case"]["page"], device="cuda") < rows[:, None])[:, :, None, None]
    return [x.index_copy_(1, dst, torch.where(mine, x.index_select(1, src), x.index_select(1, dst))) for x in s["all"]]


def _encode(x):
    """(codes, scales) of rows of float32: a block's scale is its largest element's size over 6 in e4m3, at
    least 2^-9 where that is not zero; a code is the value nearest to the quotient, ties to the even code."""
    y = x.reshape(*x.shape[:-1], -1, 16)
    a = y.abs()
    top = a.amax(-1)
    scale = torch.where(top > 0, (top / torch.full_like(top, 6.0)).clamp(2.0 ** -9, 448.0), 0.0).to(E4M3)
    by = scale.float()[..., None]
    code = (a > 0.25 * by).byte() + (a >= 0.75 * by).byte() + (a > 1.25 * by).byte() + (a >= 1.75 * by).byte() \
        + (a > 2.5 * by).byte() + (a >= 3.5 * by).byte() + (a > 5.0 * by).byte()
    code = torch.where(by > 0, code, torch.zeros_like(code)) + 8 * torch.signbit(y).byte()
    code = code.reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], scale


def _plain_append(s):
    T, page = s["case"]["tokens"], s["case"]["page"]
    slots = s["slot_map"][:T]
    kc, ks = _encode(s["k"][:T].float() * (1.0 / s["case"]["k_unit"]))
    vc, vs = _encode(s["v"][:T].float() * (1.0 / s["case"]["v_unit"]))
    where = (slots // page, slots % page)
    s["k_codes"][where], s["v_codes"][where] = kc, vc
    s["k_scales"].view(torch.uint8)[where], s["v_scales"].view(torch.uint8)[where] = ks.view(torch.uint8), vs.view(torch.uint8)
    return s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]


def _decode(codes, scales, unit, dtype=F32):
    """Values of a cache's rows."""
    both = torch.tensor([[lo, hi] for hi in VALUES + tuple(-x for x in VALUES) for lo in VALUES + tuple(-x for x in VALUES)],
                        dtype=dtype, device="cuda")
    x = both[codes.int()].reshape(*codes.shape[:-1], -1, 16)
    return x.mul_(scales.to(dtype)[..., None]).mul_(unit).reshape(*codes.shape[:-1], -1)


def _plain_fwd(s):
    case = s["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    n, group = case["n_seqs"], Hq // Hkv
    T, L, M = s["cu"][-1], s["max_kv"], s["max_q_len"]
    # all sequences side by side, as long as the longest: rows and keys past a sequence's own are masked
    pages = s["block_table"][:, :_ceil(L, page)].long().clamp(min=0)
    k = _decode(s["k_codes"][pages], s["k_scales"].view(torch.uint8)[pages].view(E4M3), case["k_unit"])
    v = _decode(s["v_codes"][pages], s["v_scales"].view(torch.uint8)[pages].view(E4M3), case["v_unit"])
    k = k.reshape(n, -1, Hkv, D)[:, :L].permute(0, 2, 3, 1)   # [n, Hkv, D, L]
    v = v.reshape(n, -1, Hkv, D)[:, :L].permute(0, 2, 1, 3)   # [n, Hkv, L, D]
    first, kv = s["cu_q"][:-1].long(), s["kv_lens"].long()
    rows = s["cu_q"][1:].long() - first
    t = torch.arange(M, device="cuda")
    q = s["q"][(first[:, None] + t).clamp(max=max(T - 1, 0))].float()  # [n, M, Hq, D]
    q = q.reshape(n, M, Hkv, group, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, group * M, D)
    z = torch.matmul(q, k).mul_(s["scale"]).reshape(n, Hkv, group, M, L)
    key = torch.arange(L, device="cuda")
    sees = kv[:, None] - rows[:, None] + t + 1 if case["causal"] else kv[:, None].expand(-1, M)
    z.masked_fill_((key >= sees[:, :, None])[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.reshape(n, Hkv, group * M, L), v).reshape(n, Hkv, group, M, D) / l
    token = torch.arange(T, device="cuda")
    of = torch.searchsorted(s["cu_q"][1:].long(), token, right=True)
    at = token - first[of]
    s["o"][:T] = o.permute(0, 3, 1, 2, 4).reshape(n, M, Hq, D)[of, at].to(s["o"].dtype)
    s["lse"][:, :T] = (m + l.log()).permute(0, 3, 1, 2, 4).reshape(n, M, Hq)[of, at].t()
    return s["o"], s["lse"]


# ------------------------------------------------------------------ work and exact values
def work(case):
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    row4 = Hkv * (D // 2 + D // 16)  # bytes of a token in 4 bits
    if case["op"] == "fork":
        kv, parents, take = _fork_plan(case)
        n, forks = len(kv), case["n_forks"]
        cols = sum(_ceil(x, page) for x in take)
        read = sum(_ceil(max(t for t, p in zip(take, parents) if p == i), page) for i in set(parents) if i >= 0)
        distinct = read  # pages whose shares change: those of the longest fork of each parent
        return {"bytes": 4 * n + 4 * forks * (2 if case["part"] else 1) + 4 * read + 4 * cols + 8 * distinct + 4 * forks
                + 12 * n + 4 * forks + 16, "flops": 0}
    if case["op"] == "free":
        kv, keep, front = _free_plan(case)
        gone = [_ceil(x, page) - _ceil(y, page) for x, y in zip(kv, keep)]
        full = max(max(front), 1)
        pages = sum(g - max(0, f - _ceil(y, page)) for g, f, y in zip(gone, front, keep)) + full  # about: each shared one once
        return {"bytes": 8 * len(kv) + 4 * sum(gone) + 8 * pages + 4 * pages + 20, "flops": 0}
    if case["op"] == "copy":
        row = row4 if case["four"] else Hkv * D * 2
        n = case["n_copies"]
        return {"bytes": 12 * (n + case["pad"]) + case["n_caches"] * n * (page + 1) * row, "flops": 0}  # half a page on average
    if case["op"] == "append":
        T = case["tokens"]
        return {"bytes": 2 * T * (2 * Hkv * D + row4) + 8 * (T + case["pad"]), "flops": 0}
    ctx, new = _lens(case)
    Hq = case["Hq"]
    T, keys = sum(new), sum(c + x for c, x in zip(ctx, new) if x)
    pairs = sum(x * c + (x * (x + 1) // 2 if case["causal"] else x * x) for c, x in zip(ctx, new))
    pages = sum(_ceil(c + x, page) for c, x in zip(ctx, new) if x)
    return {"bytes": 2 * 2 * T * Hq * D + 4 * T * Hq + 2 * keys * row4 + 4 * pages + 8 * len(new), "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    if case["op"] in ("fork", "free") or case["four"]:
        return None  # whole numbers
    s = prepare(case, seed)
    f64, page = torch.float64, case["page"]
    if case["op"] == "copy":
        x = s["all"][0].to(f64)
        for src, dst, rows in s["copies"].tolist():
            if rows > 0:
                x[:, dst, :rows] = x[:, src, :rows]
        return [x]
    if case["op"] == "append":
        slots = s["slot_map"].tolist()
        token = [i for i, x in enumerate(slots) if x >= 0]
        where = torch.tensor([(x // page, x % page) for x in slots if x >= 0], device="cuda")
        grid = [i * 2.0 ** -9 for i in range(8)] + [(1 + i / 8) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1]
        grid = torch.tensor(grid, dtype=f64, device="cuda")  # what e4m3 holds, ascending
        scales = []
        for name in ("k", "v"):
            x = s[name][token].to(f64) / case[name + "_unit"]
            want = x.unflatten(-1, (-1, 16)).abs().max(-1).values / 6
            up = torch.searchsorted(grid, want).clamp(1, len(grid) - 1)  # ties go to the even one
            low, high = grid[up - 1], grid[up]
            near = torch.where((want - low > high - want) | ((want - low == high - want) & (up % 2 == 0)), up, up - 1)
            near = torch.where((near == 0) & (want > 0), 1, near)
            full = torch.zeros(s[name + "_scales"].shape, dtype=f64, device="cuda")
            full.index_put_((where[:, 0], where[:, 1]), grid[near])
            scales.append(full)
        return None, scales[0], None, scales[1]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    group = Hq // Hkv
    T = s["q"].shape[0]
    o = torch.zeros((T, Hq, D), dtype=f64, device="cuda")
    lse = torch.zeros((Hq, T), dtype=f64, device="cuda")
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=f64, device="cuda")

    def rows_of(name, pages, rows, h):
        c = s[name + "_codes"][pages, rows, h].int()
        x = torch.empty((len(rows), D), dtype=f64, device="cuda")
        x[:, 0::2], x[:, 1::2] = value[c % 16], value[c // 16]
        by = s[name + "_scales"].view(torch.uint8)[pages, rows, h].view(E4M3).to(f64)
        return x * by.repeat_interleave(16, dim=1) * case[name + "_unit"]

    for i, (c, x) in enumerate(zip(s["ctx"], s["new"])):
        first = s["cu"][i]
        where = torch.arange(c + x, device="cuda")
        page_of = s["block_table"][i].to(I64)[where // page]
        for h in range(Hkv if x else 0):
            K, V = rows_of("k", page_of, where % page, h), rows_of("v", page_of, where % page, h)
            for b in range(0, x, 2048):
                e = min(x, b + 2048)
                seen = c + e if case["causal"] else c + x  # keys that any row of the block may see
                for hq in range(h * group, (h + 1) * group):
                    logits = s["scale"] * (s["q"][first + b:first + e, hq].to(f64) @ K[:seen].T)
                    if case["causal"]:
                        row = torch.arange(b, e, device="cuda")
                        logits[where[None, :seen] > (c + row)[:, None]] = -math.inf
                    top = logits.max(dim=1).values
                    weight = torch.exp(logits - top[:, None])
                    total = weight.sum(dim=1)
                    o[first + b:first + e, hq] = (weight @ V[:seen]) / total[:, None]
                    lse[hq, first + b:first + e] = top + torch.log(total)
    return o, lse
