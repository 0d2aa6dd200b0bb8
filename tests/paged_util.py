"""Batches on a paged latent cache for the tests: seeded host data, its device copy, and the attention's bound."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged_oracle as PO

SCALE = float(np.float32(1.0 / np.sqrt(192.0)))


def bf16(x):
    """x rounded to bf16 (nearest even), as float32."""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


class Batch:
    """B sequences of `lens` rows, the last `news` of them this call's tokens.  Rows no new token can see, pages of
    nobody and padding tokens hold NaN; table entries that must not be used hold ids far outside the pool."""

    def __init__(self, seed, e4m3, H, ps, news, lens, window=0, n_sink=0, pad=0, std=1.0, rows_std=1.0, same=None):
        rng = np.random.default_rng(seed)
        self.e4m3, self.H, self.ps, self.news, self.lens = e4m3, H, ps, list(news), list(lens)
        self.window, self.n_sink, self.B = window, n_sink, len(news)
        need = [-(-l // ps) for l in lens]
        self.n_pages = sum(need) + 2
        order = rng.permutation(self.n_pages)
        self.width = max(1, max(need)) + 1
        self.table = np.where(rng.random((self.B, self.width)) < 0.5, -1, 1 << 30).astype(np.int32)
        self.raw = np.full((self.n_pages * ps, PO.ROW8 if e4m3 else 2 * PO.ROW), 0xFF, np.uint8)   # all NaN
        self.rows, self.row_ids = [], []
        at = 0
        for b, l in enumerate(lens):
            lat = bf16(rng.standard_normal((l, PO.LAT)) * rows_std)
            rope = bf16(rng.standard_normal((l, PO.ROPE)) * rows_std)
            if same is not None and l:
                lat[:], rope[:] = lat[:1], rope[:1]
            packed = PO.pack_rows(lat, rope, e4m3)
            ids = order[at:at + need[b]]
            at += need[b]
            p = np.arange(l)
            slot = ids[p // ps] * ps + p % ps if l else np.zeros(0, int)
            see = np.zeros(l, bool)
            for i in range(news[b]):
                see |= PO.visible(l - news[b] + i, l, window, n_sink)
            self.raw[slot[see]] = packed[see]
            pages = np.unique(p[see] // ps)
            self.table[b, pages] = ids[pages]
            self.rows.append(PO.row_values(packed, e4m3))
            self.row_ids.append(slot)
        self.cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        self.q_lat = (rng.standard_normal((self.T, H, PO.LAT)) * std).astype(np.float16)
        self.q_pe = bf16(rng.standard_normal((self.T, H, PO.ROPE)) * std)
        self.q_lat[self.cu[-1]:], self.q_pe[self.cu[-1]:] = np.nan, np.nan

    def pages_dev(self):
        t = torch.from_numpy(self.raw).cuda()
        t = t if self.e4m3 else t.view(torch.float16)
        return t.reshape(self.n_pages, self.ps, -1)

    def dev(self):
        return dict(q_lat=torch.from_numpy(self.q_lat).cuda(), q_pe=torch.from_numpy(self.q_pe).bfloat16().cuda(),
                    pages=self.pages_dev(), block_table=torch.from_numpy(self.table).cuda(),
                    cu_q=torch.from_numpy(self.cu).cuda(),
                    seq_len=torch.from_numpy(np.asarray(self.lens, np.int32)).cuda())

    def ref(self):
        """(o, bound) of the cu[B] tokens.  The bound, per value, from the arithmetic: the probabilities are rounded
        once to fp16 (at most 2^-11 of each, or 2^-25 for one below fp16's normal range, where the largest is at
        least 1), scores are fp32 sums of 576 products with an error that moves a probability by less than 2^-12
        of itself at these sizes (40 accumulation steps of 2^-23 of at most ~400, times the scale 0.072), and the
        result is rounded once to fp16 (2^-11)."""
        q = np.concatenate([self.q_lat.astype(np.float64), self.q_pe.astype(np.float64)], -1)
        o, tol = [], []
        for b in range(self.B):
            if self.news[b] == 0:
                continue
            x, a, n = PO.attend(q[self.cu[b]:self.cu[b + 1]], self.rows[b], self.lens[b] - self.news[b], self.window,
                                self.n_sink, SCALE)
            o.append(x)
            tol.append((2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -11 * np.abs(x) + 2.0 ** -24
                       + 2.0 ** -25 * n[:, None, None] * np.abs(self.rows[b]).max())
        return np.concatenate(o), np.concatenate(tol)
