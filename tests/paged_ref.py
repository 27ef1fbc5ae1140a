"""Plain 64-bit implementations of the paged cache's operators, and the inputs of
their tests.

Tolerance of O, element by element.  With A = sum_j P_ij |v_j| (the exact weights):
  - P is rounded to the operands' type before the product: half a step u, so u A;
  - O is rounded once: u |O|;
  - a logit is off by at most E = 4 D 2^-24 scale |q| |k| (D products summed in fp32;
    the factor 4 for sums that truncate, one whole step of 2^-23 each, in groups), which
    changes a weight and the row's sum by a factor of at most 1 + E each: 2 E A;
  - the row sum and the product are sums of n fp32 terms: 2 n 2^-24 A;
  - the exponential, the quotient and the rescalings: 2^-19 A.
LSE is off by E + (n + 8) 2^-24 (1 + |LSE|) and the exponential's share.
u: bf16 2^-8, fp16 2^-11.
"""
import math
import random

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Batch:
    """A ragged batch over a paged cache: lens = [(cached + new keys, new rows), ...]."""

    def __init__(self, lens, Hq, Hkv, D, page, dtype=torch.bfloat16, causal=1, layout="tokens", extra_cols=2,
                 pad_rows=0, seed=0, stale=float("nan"), q_sigma=1.0, first_page=0, device="cuda", shift=0.0):
        self.lens, self.Hq, self.Hkv, self.D, self.page = lens, Hq, Hkv, D, page
        self.dtype, self.causal, self.device = dtype, causal, device
        rng = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        counts = [-(-kv // page) for kv, _ in lens]
        self.n_pages = sum(counts) + 3 + first_page
        order = list(range(first_page, self.n_pages))
        rng.shuffle(order)
        width = max(max(counts), 1) + extra_cols
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        k = torch.full((self.n_pages - first_page, page, Hkv, D), stale, dtype=dtype)
        v = torch.full_like(k, stale)
        self.dense = []
        at = 0
        for s, (kv, _) in enumerate(lens):
            pages = order[at:at + counts[s]]
            at += counts[s]
            table[s, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
            dk = torch.randn(kv, Hkv, D, generator=g).to(dtype)
            if shift:  # with q[..., 0] = 16 below: every logit is moved by about `shift`
                dk[..., 0] = shift * math.sqrt(D) / 16
            dv = torch.randn(kv, Hkv, D, generator=g).to(dtype)
            self.dense.append((dk, dv))
            for j, x in enumerate(pages):
                n = min(page, kv - j * page)
                k[x - first_page, :n] = dk[j * page:j * page + n]
                v[x - first_page, :n] = dv[j * page:j * page + n]
        self.table = table
        self.cu = np.cumsum([0] + [n for _, n in lens]).tolist()
        self.T = self.cu[-1] + pad_rows
        self.q = (q_sigma * torch.randn(max(self.T, 1), Hq, D, generator=g)).to(dtype)
        if shift:
            self.q[..., 0] = 16
        self.scale = 1 / math.sqrt(D)
        self.k_cache, self.v_cache = self._place(k, v, layout, first_page)

    def _place(self, k, v, layout, first_page):
        n, page, H, D = self.n_pages, self.page, self.Hkv, self.D
        if layout == "tokens":
            c = [torch.empty(n, page, H, D, dtype=self.dtype, device=self.device) for _ in range(2)]
        elif layout == "heads":
            c = [torch.empty(n, H, page, D, dtype=self.dtype, device=self.device).transpose(1, 2) for _ in range(2)]
        elif layout == "wide":  # a head's K and V side by side: heads 2 D apart
            x = torch.empty(n, page, H, 2 * D, dtype=self.dtype, device=self.device)
            c = [x[..., :D], x[..., D:]]
        else:  # K and V in turn
            x = torch.empty(n, 2, page, H, D, dtype=self.dtype, device=self.device)
            c = [x[:, 0], x[:, 1]]
        c[0][first_page:] = k.to(self.device)
        c[1][first_page:] = v.to(self.device)
        return c

    def on_gpu(self):
        i32 = torch.int32
        return dict(q=self.q.to(self.device), k_cache=self.k_cache, v_cache=self.v_cache,
                    block_table=self.table.to(self.device),
                    cu_q=torch.tensor(self.cu, dtype=i32, device=self.device),
                    kv_lens=torch.tensor([kv for kv, _ in self.lens], dtype=i32, device=self.device))

    def reference(self, bad_pages=()):
        """(O, LSE, bound of O's error, bound of LSE's error) in 64 bits; rows of no
        sequence hold NaN.  bad_pages: (sequence, column) entries that name no page."""
        T, Hq, D, group = max(self.T, 1), self.Hq, self.D, self.Hq // self.Hkv
        u = U[self.dtype]
        o = np.full((T, Hq, D), np.nan)
        lse = np.full((Hq, T), np.nan)
        tol_o, tol_l = np.zeros_like(o), np.zeros_like(lse)
        q = self.q.double().numpy()
        for s, (kv, n) in enumerate(self.lens):
            if n == 0:
                continue
            k, v = (x.double().numpy() for x in self.dense[s])
            key = np.arange(kv)
            there = np.ones(kv, dtype=bool)
            for bs, col in bad_pages:
                if bs == s:
                    there[col * self.page:(col + 1) * self.page] = False
            seen = np.broadcast_to(there, (n, kv)).copy()
            if self.causal:
                seen &= key[None, :] <= (kv - n) + np.arange(n)[:, None]
            a = self.cu[s]
            for h in range(Hq):
                qh, kh, vh = q[a:a + n, h], k[:, h // group], v[:, h // group]
                z = np.where(seen, self.scale * (qh @ kh.T), -np.inf) if kv else np.zeros((n, 0))
                m = z.max(axis=1, initial=-np.inf)
                w = np.exp(z - np.where(np.isneginf(m), 0, m)[:, None])
                total = w.sum(axis=1)
                with np.errstate(divide="ignore", invalid="ignore"):
                    w = np.where(total[:, None] > 0, w / total[:, None], 0)
                    lh = m + np.log(total)
                lh = np.where(total > 0, lh, -np.inf)
                oh = w @ vh
                spread = w @ np.abs(vh)
                big = 4 * D * 2.0 ** -24 * self.scale * np.linalg.norm(qh, axis=1) * \
                    np.linalg.norm(kh, axis=1).max(initial=0.0)
                o[a:a + n, h], lse[h, a:a + n] = oh, lh
                tol_o[a:a + n, h] = (u + 2 * big[:, None] + 2 * kv * 2.0 ** -24 + 2.0 ** -19) * spread + u * np.abs(oh)
                tol_l[h, a:a + n] = big + (kv + 8) * 2.0 ** -24 * (1 + np.abs(np.where(np.isneginf(lh), 0, lh))) + 2.0 ** -19
        return o, lse, tol_o, tol_l


def check(batch, o, lse, bad_pages=(), untouched=None):
    """Compare with the plain implementation; rows of no sequence have to hold `untouched`."""
    ro, rl, to, tl = batch.reference(bad_pages)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = ~np.isnan(ro)
    assert np.isfinite(o[mine]).all(), "O is not finite"
    over = np.abs(o - ro)[mine] - to[mine]
    assert over.size == 0 or over.max() <= 0, f"O off by {over.max():.3e} more than the bound"
    rows = ~np.isnan(rl)
    ninf = np.isneginf(rl) & rows
    assert np.array_equal(np.isneginf(lse) & rows, ninf), "rows without a key"
    fin = rows & ~ninf
    over = np.abs(lse[fin] - rl[fin]) - tl[fin]
    assert over.size == 0 or over.max() <= 0, f"LSE off by {over.max():.3e} more than the bound"
    if untouched is not None:
        assert (o[~mine] == untouched).all() and (lse[~rows] == untouched).all(), "rows of no sequence were written"


def plain_tables(ctx, new, free, head, table, page, max_tokens):
    """The definition, sequence by sequence: (table, cu, kv, slots, counts)."""
    table = [list(r) for r in table]
    width = len(table[0])
    cu, kv, slots, at, missing, over = [0], [], [], head, 0, 0
    for row, c, n in zip(table, ctx, new):
        c, n = max(c, 0), max(n, 0)
        for col in range(-(-c // page), -(-(c + n) // page)):
            if col >= width:
                continue
            if at < len(free):
                row[col] = free[at]
                at += 1
            else:
                row[col] = -1
                missing += 1
        over += -(-(c + n) // page) > width
        for pos in range(c, c + n):
            x = row[pos // page] if pos // page < width else -1
            slots.append(x * page + pos % page if x >= 0 else -1)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    return table, cu, kv, slots, [cu[-1], at, missing, over]
