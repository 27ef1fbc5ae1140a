"""Plain implementations of the cache in 4 bits and of the bookkeeping of shared pages, and
the inputs of their tests.

Tolerance of O, element by element, as in paged_ref.py but for the types of the operands.  With
A = sum_j P_ij |v_j| and B = sum_j |v_j| over the seen keys:
  - K, V are exact in fp16; q in bf16 becomes fp16 off by at most 2^-39 of its row's largest element,
    which moves a logit by at most F = D 2^-39 scale max|q| max|k|;
  - P is rounded to fp16 before its product: half a step, 2^-11 A, or 2^-25 B where it is below
    fp16's normal numbers (weights are relative to a maximum of at most 1, which is in the sum);
  - O is rounded once to its type: u |O|;
  - a logit is off by at most E = 4 D 2^-24 scale |q| |k| + F: 2 E A;
  - the row sum and the product are sums of n fp32 terms: 2 n 2^-24 A;
  - the exponential, the quotient, the rescalings and the products with scales and units: 2^-19 A.
LSE is off by E + (n + 8) 2^-24 (1 + |LSE|) and the exponential's share.
"""
import math
import random

import numpy as np
import torch

from paged_ref import U, Batch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values():
    """Values of the 256 bytes, NaN at 0x7f and 0xff."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_values()


def encode(x, inv):
    """(codes [.., D / 2], scales [.., D / 16]) as uint8 of float32 rows, element by element."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        y = x * np.float32(inv)
    blocks = y.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    big = np.float32(np.finfo(np.float32).max)
    blocks = np.where(np.isnan(blocks), big, np.clip(blocks, -big, big)).astype(np.float32)
    with np.errstate(all="ignore"):
        want = (np.abs(blocks).max(-1) / np.float32(6)).astype(np.float64)
    grid = E4M3[:127]  # ascending; the even byte takes ties
    up = np.clip(np.searchsorted(grid, want), 1, 126)
    low, high = grid[up - 1], grid[up]
    byte = np.where((want - low > high - want) | ((want - low == high - want) & (up % 2 == 0)), up, up - 1)
    byte = np.where((byte == 0) & (np.abs(blocks).max(-1) > 0), 1, byte)
    s = grid[byte].astype(np.float32)[..., None]
    with np.errstate(all="ignore"):
        t = np.where(s > 0, np.abs(blocks) / np.where(s > 0, s, 1), 0).astype(np.float32)
    code = np.zeros(t.shape, dtype=np.uint8)
    for i, border in enumerate((.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (t > border) if i % 2 == 0 else (t >= border)  # ties to the even code
    code |= np.signbit(blocks).astype(np.uint8) << 3
    code = code.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), byte.astype(np.uint8)


def decode(codes, scales, unit):
    """Values in 64 bits."""
    codes = np.asarray(codes)
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], codes.shape[-1] // 8, 16)
    return (v * E4M3[np.asarray(scales)][..., None]).reshape(*codes.shape[:-1], 2 * codes.shape[-1]) * unit


def place(shape, layout, fill, device="cuda"):
    """Two caches [n_pages, page, Hkv, x] of bytes, `fill` where nothing is written, in one layout."""
    n, page, H, x = shape
    full = lambda *s: torch.full(s, fill, dtype=torch.uint8, device=device)  # noqa: E731
    if layout == "tokens":
        return [full(n, page, H, x) for _ in range(2)]
    if layout == "heads":
        return [full(n, H, page, x).transpose(1, 2) for _ in range(2)]
    if layout == "wide":  # a head's K and V side by side
        y = full(n, page, H, 2 * x)
        return [y[..., :x], y[..., x:]]
    y = full(n, 2, page, H, x)  # K and V in turn
    return [y[:, 0], y[:, 1]]


class Batch4(Batch):
    """A ragged batch over a cache in 4 bits.  Unwritten rows hold scales that are NaN."""

    def __init__(self, lens, Hq, Hkv, D, page, dtype=torch.bfloat16, layout="tokens", k_unit=1.0, v_unit=1.0, sigma=1.0,
                 first_page=0, stale=0x7f, **kw):
        super().__init__(lens, Hq, Hkv, D, page, dtype, stale=0.0, device="cpu", **kw)
        self.k_unit, self.v_unit, self.device = k_unit, v_unit, "cuda"
        n = self.n_pages + first_page
        codes, scales = place((n, page, Hkv, D // 2), layout, 0x77), place((n, page, Hkv, D // 16), layout, stale)
        if first_page:
            self.table = torch.where(self.table >= 0, self.table + first_page, self.table)
        self.n_pages = n
        host = [[torch.full((n - first_page, page, Hkv, D // 2), 0x77, dtype=torch.uint8) for _ in range(2)],
                [torch.full((n - first_page, page, Hkv, D // 16), stale, dtype=torch.uint8) for _ in range(2)]]
        for s, (kv, _) in enumerate(lens):
            both = []
            for i, unit in enumerate((k_unit, v_unit)):
                c, b = encode(sigma * unit * self.dense[s][i].float().numpy(), 1.0 / unit)
                for j in range(-(-kv // page)):
                    m, at = min(page, kv - j * page), int(self.table[s, j]) - first_page
                    host[0][i][at, :m] = torch.from_numpy(c[j * page:j * page + m])
                    host[1][i][at, :m] = torch.from_numpy(b[j * page:j * page + m])
                both.append(torch.from_numpy(decode(c, b, unit)))
            self.dense[s] = tuple(both)
        for x, y in zip(codes + scales, host[0] + host[1]):
            x[first_page:] = y.to("cuda")
        self.k_codes, self.v_codes = codes
        self.k_scales, self.v_scales = scales
        self.scale = 1 / (math.sqrt(D) * k_unit * sigma)

    def on_gpu(self):
        i32 = torch.int32
        return dict(q=self.q.cuda(), k_codes=self.k_codes, k_scales=self.k_scales, v_codes=self.v_codes,
                    v_scales=self.v_scales, block_table=self.table.cuda(),
                    cu_q=torch.tensor(self.cu, dtype=i32, device="cuda"),
                    kv_lens=torch.tensor([kv for kv, _ in self.lens], dtype=i32, device="cuda"))

    def reference(self, bad_pages=()):
        T, Hq, D, group = max(self.T, 1), self.Hq, self.D, self.Hq // self.Hkv
        u, up = U[self.dtype], 2.0 ** -11
        o, lse = np.full((T, Hq, D), np.nan), np.full((Hq, T), np.nan)
        tol_o, tol_l = np.zeros_like(o), np.zeros_like(lse)
        q = self.q.double().numpy()
        for s, (kv, n) in enumerate(self.lens):
            if n == 0:
                continue
            k, v = (np.asarray(x) for x in self.dense[s])
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
                oh, spread, mass = w @ vh, w @ np.abs(vh), seen @ np.abs(vh)
                big = 4 * D * 2.0 ** -24 * self.scale * np.linalg.norm(qh, axis=1) * np.linalg.norm(kh, axis=1).max(initial=0.0)
                big += D * 2.0 ** -39 * self.scale * np.abs(qh).max(axis=1) * np.abs(kh).max(initial=0.0)
                o[a:a + n, h], lse[h, a:a + n] = oh, lh
                tol_o[a:a + n, h] = (up + 2 * big[:, None] + 2 * kv * 2.0 ** -24 + 2.0 ** -19) * spread + \
                    2.0 ** -25 * mass + u * np.abs(oh)
                tol_l[h, a:a + n] = big + (kv + 8) * 2.0 ** -24 * (1 + np.abs(np.where(np.isneginf(lh), 0, lh))) + 2.0 ** -19
        return o, lse, tol_o, tol_l


def plain_fork(parents, lens, kv, free, head, table, page, shares):
    """The definition, row by row: (kv, table, shares, copies, counts)."""
    n, width, n_pages = len(parents), len(table[0]), len(shares)
    table, kv, shares = [list(r) for r in table], list(kv), list(shares)
    parent = [p if 0 <= p < n and p != i else -1 for i, p in enumerate(parents)]
    copies, forks, missing, left, at = [], 0, 0, 0, head
    for i, p in enumerate(parent):
        copies.append([-1, -1, 0])
        if p < 0:
            continue
        if parent[p] >= 0:
            left += 1
            continue
        forks += 1
        t = min(max(kv[p], 0), width * page)
        if lens is not None:
            t = min(t, max(lens[i], 0))
        kv[i] = t
        for col in range(t // page):
            x = table[i][col] = table[p][col]
            if 0 <= x < n_pages:
                shares[x] += 1
        if t % page:
            src = table[p][t // page]
            if not 0 <= src < n_pages:
                table[i][t // page] = src
            elif at < len(free):
                table[i][t // page] = free[at]
                copies[i] = [src, free[at], t % page]
                at += 1
            else:
                table[i][t // page] = -1
                missing += 1
    return kv, table, shares, copies, [forks, at, missing, left]


def plain_free(kv, keep, table, page, shares, free, head):
    """The definition, row by row: (shares, free, counts)."""
    width, n_pages, n_free = len(table[0]), len(shares), len(free)
    shares, free = list(shares), list(free)
    for row, a, b in zip(table, kv, keep):
        a, b = min(max(a, 0), width * page), max(b, 0)
        for col in range(-(-b // page), -(-a // page)):
            if 0 <= row[col] < n_pages:
                shares[row[col]] -= 1
    freed = [x for x in range(n_pages) if shares[x] < 0]
    for x in freed:
        shares[x] = 0
    cut = 0
    for row, a, b in zip(table, kv, keep):
        a, b = min(max(a, 0), width * page), max(b, 0)
        if b < a and b % page and 0 <= row[b // page] < n_pages:
            cut += shares[row[b // page]] > 0
    head = min(max(head, 0), n_free)
    fit = min(len(freed), head)
    if fit:
        free[head - fit:head] = freed[len(freed) - fit:]
    return shares, free, [fit, head - fit, len(freed) - fit, cut]


def random_rows(rng, n, page, hi, width, n_pages, full=0.2):
    """Rows of distinct pages and their tokens."""
    kv = [rng.choice([0, rng.randint(0, hi), rng.randint(0, hi) // page * page]) for _ in range(n)]
    pages = list(range(n_pages))
    rng.shuffle(pages)
    table, at = [], 0
    for x in kv:
        m = -(-x // page)
        table.append(pages[at:at + m] + [-7] * (width - m))
        at += m
    assert at <= n_pages
    return kv, table, pages[at:]
