"""Pools, tables and 64-bit statements of the calls over paged caches, for the tests."""

from __future__ import annotations

import math

import numpy as np
import torch

from tests import attend_ref as ref

D = 128


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_status():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


class Pool:
    """Slots of `batch` sequences on random pages (page None: dense caches of `cap` slots)."""

    def __init__(self, batch, kv, slots, page, seed, extra=3):
        self.batch, self.kv, self.page = batch, kv, page
        rs = np.random.RandomState(seed)
        if page is None:
            self.size, self.pages, self.table = max(max(slots) + 3, 2), batch, None
            self.where = [np.full(self.size, b) for b in range(batch)], [np.arange(self.size)] * batch
            return
        self.size = page
        used = [-(-n // page) for n in slots]
        self.pages = sum(used) + extra
        order, at = rs.permutation(self.pages), 0
        table = np.full((batch, max(used + [1]) + 1), -1, np.int32)  # entries behind the last page name none
        pg, place = [], []
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n]
            at += n
            pg.append(np.repeat(table[b, :n], page))
            place.append(np.tile(np.arange(page), n))
        self.where = pg, place
        self.table = torch.from_numpy(table).cuda()

    def config(self, bkv, heads, **over):
        cap = self.size if self.table is None else self.size * self.table.shape[1]
        args = dict(heads=heads, kv_heads=self.kv, d=D, budget=1, period=16, prefix=0, recent=0, layers=1, batch=self.batch,
                    max_cache=max(cap, 2), rope_theta=1e6)
        args.update(over)
        return bkv.make_config(**args)

    def shape(self):
        return (self.pages, self.kv, self.size)

    def at(self, b, n, start=0):
        """Pages and places of slots [start, n) of sequence b."""
        return (torch.from_numpy(np.asarray(self.where[0][b][start:n]).astype(np.int64)).cuda(),
                torch.from_numpy(np.asarray(self.where[1][b][start:n]).astype(np.int64)).cuda())

    def get(self, pool, b, n):
        """Slots [0, n) of sequence b, [kv][n]..."""
        page, place = self.at(b, n)
        return pool[page, :, place].transpose(0, 1)

    def put(self, pool, b, n, rows, start=0):
        page, place = self.at(b, n, start)
        pool[page, :, place] = rows.transpose(0, 1).to(pool.dtype)

    def fresh(self, slots, seed, scale=1.0, fill=math.nan):
        """A bf16 pool with random rows in the sequences' slots and `fill` everywhere else."""
        pool = torch.full(self.shape() + (D,), fill, dtype=torch.bfloat16, device="cuda")
        for b, n in enumerate(slots):
            if n:
                self.put(pool, b, n, randn((self.kv, n, D), seed + b, scale))
        return pool


def probabilities(q, K, see):
    """p [n][H][L] in float64 and a relative bound per (row, head), for weights: a logit is off
    by e (as in attend_ref), the log-sum-exp by its own bound, their difference and its
    exponential by (|l| + |lse| + 4) 2^-22."""
    n, H, _ = q.shape
    kv, L = K.shape[:2]
    G = H // kv
    _, lse, _, lse_tol = ref.attention(q, K, torch.zeros_like(K), see)
    p = torch.zeros((n, H, L), dtype=torch.float64, device=q.device)
    rel = torch.zeros((n, H), dtype=torch.float64, device=q.device)
    for h in range(H):
        x, k = q[:, h].double(), K[h // G].double()
        l = (x @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf)
        p[:, h] = torch.exp(l - lse[:, h:h + 1]).masked_fill(~see, 0.0)
        size = (x.abs() @ k.abs().T / math.sqrt(D)).masked_fill(~see, 0.0).amax(dim=1)
        top = l.masked_fill(~see, 0.0).abs().amax(dim=1)
        rel[:, h] = 127 * 2.0 ** -23 * size + lse_tol[:, h] + (2 * top + lse[:, h].abs() + 4) * 1.4427 * 2.0 ** -22
    return p, rel, lse


def weight_sums(p, rel, kv):
    """Sums over rows and the KV heads' query heads, [kv][L], and their bound: every term's own,
    the sum's n G 2^-23, and what ex2 flushes to zero."""
    n, H, L = p.shape
    s = p.view(n, kv, H // kv, L).sum(dim=(0, 2))
    tol = (p * rel[..., None]).view(n, kv, H // kv, L).sum(dim=(0, 2)) + s * (n * H // kv) * 2.0 ** -23 + n * H * 2.0 ** -126
    return s, tol


def keep_set(w, budget, prefix, recent):
    """The eviction's keep set of one unit's weights (a numpy float32 array), ascending."""
    n = len(w)
    middle = np.arange(prefix, n - recent)
    key = np.where(np.isnan(w[middle]), -np.inf, w[middle].astype(np.float64))
    below = np.isnan(w[middle])  # NaN behind -inf
    order = np.lexsort((middle, below, -key))
    best = middle[order][:budget - prefix - recent]
    return np.sort(np.concatenate([np.arange(prefix), best, np.arange(n - recent, n)]))


def order_free_layout(kept, budget):
    layout = np.arange(budget)
    layout[np.setdiff1d(layout, kept)] = kept[kept >= budget]
    return layout
