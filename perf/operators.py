"""Cases that measure the paged key/value cache of libattn: the tables that say where each token lives,
the write of new keys and values, and attention of new tokens over the cache.

`own = False` computes the operators in plain torch; `own = True` calls libattn.
"""
import math
import random

import torch

own = False

F32 = torch.float32


# ------------------------------------------------------------------ cases
def listed():
    """What each stands for in real use is said above it."""
    return [
        # one decode step's bookkeeping: every running request grows by one token
        _case("tables_decode_64", op="tables", n_seqs=64, n_chunks=0, page=16, ctx_lo=100, ctx_hi=8000, max_pages=640),
        # a large scheduler step: 1024 requests, most of them with a chunk of their prompt, a padded token count
        _case("tables_chunks_1024", op="tables", n_seqs=1024, n_chunks=900, q_lo=1, q_hi=256, page=64, ctx_lo=0,
              ctx_hi=30000, max_pages=513, pad=1000),
        # the same two steps' cache writes: 64 single tokens cut out of a fused projection ...
        _case("append_decode_64", op="append", tokens=64, Hq=32, Hkv=8, D=128, page=16, n_pages=4096, fused=True),
        # ... and the prompts of many requests at once, padded to a fixed count
        _case("append_prompts_65000", op="append", tokens=65000, Hq=16, Hkv=16, D=64, page=128, n_pages=600, f16=True,
              pad=536),
        # one user, one token, a short context: latency
        _case("decode_1x1000", op="fwd", n_seqs=1, Hq=32, Hkv=8, ctx_lo=1000, ctx_hi=1000, page=16),
        # few users with long contexts, one K/V head: the benchmark's decode shape, in pages
        _case("decode_8x32768", op="fwd", n_seqs=8, Hq=8, Hkv=1, ctx_lo=32767, ctx_hi=32767, page=64),
        # a decode batch of unlike lengths, captured for 64 requests of which 48 are there
        _case("decode_ragged_48", op="fwd", n_seqs=64, n_empty=16, Hq=64, Hkv=8, ctx_lo=300, ctx_hi=8000, page=16,
              pad=16),
        # drafted tokens being verified: five new tokens a request
        _case("verify_16x5", op="fwd", n_seqs=16, n_chunks=16, q_lo=5, q_hi=5, Hq=32, Hkv=8, D=64, ctx_lo=2000,
              ctx_hi=6000, page=32, f16=True),
        # one scheduler step that mixes prompt chunks with decoding requests; pages stored head by head
        _case("mixed_4_chunks_36", op="fwd", n_seqs=40, n_chunks=4, q_lo=100, q_hi=512, Hq=32, Hkv=8, ctx_lo=500,
              ctx_hi=6000, page=16, heads_first=True),
        # the benchmark's chunked prefill, in pages
        _case("chunk_512x32768", op="fwd", n_seqs=1, n_chunks=1, q_lo=512, q_hi=512, Hq=64, Hkv=8, ctx_lo=32256,
              ctx_hi=32256, page=64),
        # rescoring of texts of odd lengths with every key visible, one head a key head
        _case("rescore_mha_d64", op="fwd", n_seqs=6, n_chunks=6, q_lo=700, q_hi=1999, Hq=16, Hkv=16, D=64, ctx_lo=0,
              ctx_hi=0, page=48, causal=0, f16=True),
        # whole prompts into an empty cache: the benchmark's grouped-head shape
        _case("prefill_2x8192", op="fwd", n_seqs=2, n_chunks=2, q_lo=8192, q_hi=8192, Hq=32, Hkv=8, ctx_lo=0, ctx_hi=0,
              page=128),
    ]


def _case(name, **kw):
    base = dict(name=name, op="fwd", n_seqs=1, n_chunks=0, n_empty=0, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=0, Hq=32, Hkv=8,
                D=128, page=16, causal=1, f16=False, pad=0, heads_first=False, fused=False, tokens=0, n_pages=0,
                max_pages=0)
    base.update(kw)
    return base


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the same ranges."""
    what = rng.choice(["tables", "append", "decode", "decode", "verify", "mixed", "chunk", "chunk", "prefill"])
    f16 = rng.random() < 0.4
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    heads_first = rng.random() < 0.3
    if what == "tables":
        n = _log(rng, 1, 1024)
        hi = _log(rng, 100, 30000)
        return _case("", op="tables", n_seqs=n, n_chunks=rng.randint(0, n), q_lo=1, q_hi=_log(rng, 2, 256), page=page,
                     ctx_lo=0, ctx_hi=hi, max_pages=(hi + 256) // page + rng.randint(1, 40), pad=rng.randint(0, 500))
    if what == "append":
        t = _log(rng, 1, 65000 if D * Hkv <= 1024 else 20000)
        return _case("", op="append", tokens=t, Hq=2 * Hkv, Hkv=Hkv, D=D, page=page, n_pages=t // page + rng.randint(2, 90),
                     f16=f16, pad=rng.randint(0, 60), fused=rng.random() < 0.5, heads_first=heads_first)
    kw = dict(op="fwd", Hq=Hkv * group, Hkv=Hkv, D=D, page=page, f16=f16, heads_first=heads_first)
    if what == "decode":
        n = _log(rng, 1, 128)
        hi = _log(rng, 64, min(60000, 2_000_000 // (n * Hkv)))
        return _case("", n_seqs=n + 3, n_empty=3, ctx_lo=hi // 8, ctx_hi=hi, pad=rng.randint(0, 20), **kw)
    if what == "verify":
        n = _log(rng, 1, 64)
        hi = _log(rng, 64, min(30000, 1_000_000 // (n * Hkv)))
        return _case("", n_seqs=n, n_chunks=n, q_lo=2, q_hi=rng.randint(2, 9), ctx_lo=hi // 4, ctx_hi=hi, **kw)
    if what == "mixed":
        n = rng.randint(4, 40)
        return _case("", n_seqs=n, n_chunks=rng.randint(1, 4), q_lo=10, q_hi=rng.randint(16, 700), ctx_lo=0,
                     ctx_hi=_log(rng, 100, 6000), pad=rng.randint(0, 9), **kw)
    if what == "chunk":
        q = _log(rng, 16, 1024)
        return _case("", n_seqs=1, n_chunks=1, q_lo=q, q_hi=q, ctx_lo=0, ctx_hi=_log(rng, 100, 16000), **kw)
    n = rng.randint(1, 4)
    return _case("", n_seqs=n, n_chunks=n, q_lo=1, q_hi=_log(rng, 100, 4000), causal=rng.randint(0, 1), **kw)


def _lens(case):
    """Cached and new tokens of every sequence: lists that depend on the case alone."""
    r = random.Random("%(n_seqs)d %(n_chunks)d %(q_lo)d %(q_hi)d %(ctx_lo)d %(ctx_hi)d" % case)
    n = case["n_seqs"]
    q = [r.randint(case["q_lo"], case["q_hi"]) if i < case["n_chunks"] else 1 for i in range(n)]
    q = [0 if i >= n - case["n_empty"] else x for i, x in enumerate(q)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    both = [(c, x) if x else (0, 0) for c, x in zip(ctx, q)]
    live = both[:n - case["n_empty"]]
    r.shuffle(live)
    both[:len(live)] = live
    return [b[0] for b in both], [b[1] for b in both]


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, g):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _caches(case, n_pages, dtype, g):
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    if case["heads_first"]:  # the same 4-d view, stored [page, head, token, D]
        return tuple(_normal((n_pages, Hkv, page, D), dtype, g).transpose(1, 2) for _ in range(2))
    return tuple(_normal((n_pages, page, Hkv, D), dtype, g) for _ in range(2))


def prepare(case, seed):
    g = _gen(seed)
    dtype = torch.float16 if case["f16"] else torch.bfloat16
    page, Hq, Hkv, D = case["page"], case["Hq"], case["Hkv"], case["D"]
    s = {"case": case}
    if case["op"] == "append":
        T, n_pages = case["tokens"], case["n_pages"]
        s["k_cache"], s["v_cache"] = _caches(case, n_pages, dtype, g)
        rows = T + case["pad"]
        if case["fused"]:  # q, k and v of one projection
            x = _normal((rows, Hq + 2 * Hkv, D), dtype, g)
            s["k"], s["v"] = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["k"], s["v"] = _normal((rows, Hkv, D), dtype, g), _normal((rows, Hkv, D), dtype, g)
        slots = torch.randperm(n_pages * page, device="cuda", generator=g)[:rows]
        slots[T:] = -1  # the rows that pad the batch
        s["slot_map"] = slots
        return s
    ctx, new = _lens(case)
    n = len(ctx)
    s["ctx"], s["new"] = ctx, new
    have = [_ceil(c, page) for c in ctx]
    want = [_ceil(c + x, page) for c, x in zip(ctx, new)]
    if case["op"] == "tables":
        n_free = sum(w - h for w, h in zip(want, have)) + 100
        pages = torch.randperm(sum(have) + n_free, device="cuda", generator=g, dtype=torch.int32)
        s["block_table"] = _table(pages[n_free:], have, case["max_pages"])
        s["free_pages"] = pages[:n_free].contiguous()
        s["ctx_lens"], s["new_lens"] = _ints(ctx), _ints(new)
        s["max_tokens"] = sum(new) + case["pad"]
        return s
    n_pages = sum(want) + 7
    pages = torch.randperm(n_pages, device="cuda", generator=g, dtype=torch.int32)
    s["block_table"] = _table(pages, want, max(want) + 3)
    s["k_cache"], s["v_cache"] = _caches(case, n_pages, dtype, g)
    T = sum(new) + case["pad"]
    s["q"] = _normal((T, Hq, D), dtype, g)
    s["scale"] = 1.0 / math.sqrt(D)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu"] = cu
    s["cu_q"], s["kv_lens"] = _ints(cu), _ints([c + x for c, x in zip(ctx, new)])
    s["max_q_len"] = max(new)
    s["o"] = torch.zeros((T, Hq, D), dtype=dtype, device="cuda")
    s["lse"] = torch.zeros((Hq, T), dtype=F32, device="cuda")
    if own:
        import attention_forward_11_gb300 as fa
        size = fa.attn_paged_fwd_workspace_size(T, s["max_q_len"], Hq, Hkv, D, page)
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


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


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import attention_forward_11_gb300 as fa
        if op == "tables":
            cu, kv, slots, counts = fa.attn_paged_tables(s["ctx_lens"], s["new_lens"], s["free_pages"], s["block_table"],
                                                         s["case"]["page"], s["max_tokens"])
            return s["block_table"], cu, kv, slots, counts
        if op == "append":
            fa.attn_paged_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"])
            return s["k_cache"], s["v_cache"]
        return fa.attn_paged_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"], s["kv_lens"],
                                 max_q_len=s["max_q_len"], causal=s["case"]["causal"], scale=s["scale"], o=s["o"],
                                 lse=s["lse"], workspace=s["workspace"])
    return {"tables": _plain_tables, "append": _plain_append, "fwd": _plain_fwd}[op](s)


def _plain_tables(s):
    page, table, free = s["case"]["page"], s["block_table"], s["free_pages"]
    ctx, new = s["ctx_lens"].long(), s["new_lens"].long()
    n, width = table.shape
    cu = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.cumsum(new, 0)
    kv = ctx + new
    have = ((ctx + page - 1) // page).clamp(max=width)
    want = ((kv + page - 1) // page).clamp(max=width)
    need = want - have
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(width, device="cuda")
    at = first[:, None] + cols - have[:, None]
    fresh = torch.where(at < len(free), free[at.clamp(0, len(free) - 1)], -1)
    table.copy_(torch.where((cols >= have[:, None]) & (cols < want[:, None]), fresh, table))
    token = torch.arange(s["max_tokens"], device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    there = seq < n
    seq = seq.clamp(max=n - 1)
    pos = ctx[seq] + token - cu[seq]
    col = pos // page
    entry = table[seq, col.clamp(0, width - 1)].long()
    slots = torch.where(there & (col < width) & (entry >= 0), entry * page + pos % page, -1)
    asked = need.sum()
    taken = asked.clamp(max=len(free))
    over = ((kv + page - 1) // page > width).sum()
    counts = torch.stack([cu[-1], taken, asked - taken, over]).int()
    return table, cu.int(), kv.int(), slots, counts


def _plain_append(s):
    T = s["case"]["tokens"]
    slots, page = s["slot_map"][:T], s["case"]["page"]
    for new, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        cache[slots // page, slots % page] = new[:T]
    return s["k_cache"], s["v_cache"]


def _plain_fwd(s):
    case = s["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    for i, (c, x) in enumerate(zip(s["ctx"], s["new"])):
        if x == 0:
            continue
        kv, a = c + x, s["cu"][i]
        pages = s["block_table"][i, :_ceil(kv, page)].long()
        k = s["k_cache"][pages].reshape(-1, Hkv, D)[:kv].float().permute(1, 2, 0)      # [Hkv, D, kv]
        v = s["v_cache"][pages].reshape(-1, Hkv, D)[:kv].float().permute(1, 0, 2)      # [Hkv, kv, D]
        q = s["q"][a:a + x].float().reshape(x, Hkv, -1, D).permute(1, 2, 0, 3)         # [Hkv, group, x, D]
        z = torch.matmul(q.reshape(Hkv, -1, D), k).mul_(s["scale"]).reshape(Hkv, -1, x, kv)
        if case["causal"]:
            t = torch.arange(x, device="cuda")[:, None]
            z.masked_fill_(torch.arange(kv, device="cuda") > c + t, -math.inf)
        m = z.amax(-1, keepdim=True)
        p = z.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.reshape(Hkv, -1, kv), v).reshape(Hkv, -1, x, D) / l
        s["o"][a:a + x] = o.permute(2, 0, 1, 3).reshape(x, Hq, D).to(s["o"].dtype)
        s["lse"][:, a:a + x] = (m + l.log()).reshape(Hq, x)
    return s["o"], s["lse"]


# ------------------------------------------------------------------ work and exact values
def work(case):
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (2 * 2 * case["Hkv"] * case["D"] * 2) + 8 * (case["tokens"] + case["pad"]), "flops": 0}
    ctx, new = _lens(case)
    n, page = len(ctx), case["page"]
    if case["op"] == "tables":
        fresh = sum(_ceil(c + x, page) - _ceil(c, page) for c, x in zip(ctx, new))
        kept = sum(1 for c, x in zip(ctx, new) if c % page and x)
        return {"bytes": 8 * n + 4 * (fresh + kept) + 4 * (2 * n + 1) + 4 * fresh + 8 * (sum(new) + case["pad"]) + 16,
                "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T, keys = sum(new), sum(c + x for c, x in zip(ctx, new) if x)
    pairs = sum(x * c + (x * (x + 1) // 2 if case["causal"] else x * x) for c, x in zip(ctx, new))
    pages = sum(_ceil(c + x, page) for c, x in zip(ctx, new) if x)
    return {"bytes": 2 * 2 * T * Hq * D + 4 * T * Hq + 2 * 2 * keys * Hkv * D + 4 * pages + 8 * n,
            "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "append":
        flat = s["slot_map"].tolist()
        where = torch.tensor([(j, x // page, x % page) for j, x in enumerate(flat) if x >= 0], device="cuda")
        for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            cache.index_put_((where[:, 1], where[:, 2]), rows.index_select(0, where[:, 0]))
        return s["k_cache"].double(), s["v_cache"].double()
    if case["op"] == "tables":
        free = s["free_pages"].tolist()
        table = s["block_table"].tolist()
        cu, kv, slots, at = [0], [], [], 0
        for row, c, x in zip(table, s["ctx"], s["new"]):
            for pos in range(c, c + x):
                col, off = divmod(pos, page)
                if off == 0:
                    row[col] = free[at]
                    at += 1
                slots.append(row[col] * page + off)
            cu.append(cu[-1] + x)
            kv.append(c + x)
        slots += [-1] * (s["max_tokens"] - len(slots))
        return torch.tensor(table), torch.tensor(cu), torch.tensor(kv), torch.tensor(slots), torch.tensor([cu[-1], at, 0, 0])
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    group = Hq // Hkv
    T = s["q"].shape[0]
    o = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((Hq, T), dtype=torch.float64, device="cuda")
    f64 = torch.float64
    for i, (c, x) in enumerate(zip(s["ctx"], s["new"])):
        first = s["cu"][i]
        where = torch.arange(c + x, device="cuda")
        page_of = s["block_table"][i].to(torch.int64)[where // page]
        for h in range(Hkv if x else 0):
            K = s["k_cache"][page_of, where % page, h].to(f64)
            V = s["v_cache"][page_of, where % page, h].to(f64)
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
