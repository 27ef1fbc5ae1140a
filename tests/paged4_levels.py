"""A batch over the cache in 4 bits with two sizes of logits and of values, for tests of weights and sums that lie
far apart."""
import math
import random

import numpy as np
import torch

from paged4_ref import Batch4, decode, encode


class Levels(Batch4):
    """Logits are gap * ln 2 for the keys that high(j) names and 0 for the others, whatever the row (times q0); the values are
    v_high and v_low (times v_unit)."""

    def __init__(self, lens, Hkv, group, D, dtype, high, gap, v_high, v_low, v_unit=1.0, q0=1.0):
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.dtype, self.causal = lens, Hkv * group, Hkv, D, 16, dtype, 1
        self.k_unit, self.v_unit, self.device = 1.0, v_unit, "cuda"
        counts = [-(-kv // 16) for kv, _ in lens]
        self.n_pages = sum(counts) + 3
        order = list(range(self.n_pages))
        random.Random(D).shuffle(order)
        self.table = torch.full((len(lens), max(counts) + 2), -1, dtype=torch.int32)
        self.cu = np.cumsum([0] + [n for _, n in lens]).tolist()
        self.T = self.cu[-1]
        self.q = torch.zeros(self.T, self.Hq, D, dtype=dtype)
        self.q[..., 0] = q0
        self.scale = gap * math.log(2) / 6
        rows = np.zeros((2, 2, D), np.float32)  # K and V of low and high keys
        rows[0, 1, 0] = 6.0
        rows[1, 0], rows[1, 1] = v_low, v_high
        codes, scales = encode(rows, 1.0)
        values = [decode(codes[0], scales[0], 1.0), decode(codes[1], scales[1], v_unit)]
        host = [np.full((self.n_pages, 16, Hkv, n), fill, np.uint8) for n, fill in ((D // 2, 0x77), (D // 16, 0x7f)) * 2]
        self.dense, at = [], 0
        for s, (kv, _) in enumerate(lens):
            which = np.array([high(j) for j in range(kv)], dtype=int)
            pages = order[at:at + counts[s]]
            at += counts[s]
            self.table[s, :counts[s]] = torch.tensor(pages, dtype=torch.int32)
            for j, page in enumerate(pages):
                w = which[16 * j:16 * j + 16]
                for x, bytes_of in zip(host, (codes[0], scales[0], codes[1], scales[1])):
                    x[page, :len(w)] = bytes_of[w][:, None]
            self.dense.append(tuple(np.broadcast_to(v[which][:, None], (kv, Hkv, D)) for v in values))
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = (torch.from_numpy(x).cuda() for x in host)
