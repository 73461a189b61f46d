"""Routings of the per-rank stage 2 with expert order, worked out on the host (not collected by pytest).

Bounds: an fp32 fma chain of m terms from zero is within m 2^-24 of its terms' magnitudes from the exact sum, and its
rounding to bf16 within 2^-8 of the value; a dot product of H terms in any order within H 2^-24 of their magnitudes.
"""
from __future__ import annotations

import numpy as np
import torch

from expert_util import BF16, D, HALF, near, normal
from gpu_util import ep

STALE = -7.25


class Ranks:
    """A group with the per-rank stage 2 and expert order, a handle, and its rows and places."""

    def __init__(self, S=1, T=40, E=16, K=4, H=256, nodes=2, per_node=2, payload="bf16", seed=0, topk=None, **over):
        rng = np.random.default_rng(seed)
        self.S, self.T, self.E, self.K, self.H = S, T, E, K, H
        self.n = n = S * T
        R = nodes * per_node
        if topk is None:
            topk = np.argsort(rng.random((n, E)), axis=1)[:, :K].astype(np.int32)
        self.topk = topk
        cfg = dict(mode="ht", num_nodes=nodes, ranks_per_node=per_node, num_experts=E, top_k=K, max_nodes_per_token=0,
                   hidden=H, max_tokens_per_rank=max(T, 1), num_src_ranks=S, payload=payload, ht_stage2="rank_sorted")
        cfg.update(over)
        self.group = ep.ep_create_group(**cfg)
        self.idx = torch.from_numpy(np.ascontiguousarray(topk)).cuda()
        self.handle = ep.ep_create_handle(self.group, self.idx)
        self.place = np.full((n, K), -1, np.int64)
        self.row = np.full((n, K), -1, np.int64)
        self.count = np.zeros(E, np.int64)
        self.rank_count = np.zeros(R, np.int64)
        valid = np.zeros((n, K), bool)
        for i in range(n):
            for k in range(K):
                e = topk[i, k]
                valid[i, k] = 0 <= e < E and e not in topk[i, :k]
        at = 0
        for e in range(E):
            for i, k in zip(*np.nonzero(valid & (topk == e))):
                self.place[i, k] = at
                at += 1
                self.count[e] += 1
        self.places = at
        at = 0
        for d in range(R):
            on = valid & (topk // (E // R) == d)
            for i in np.flatnonzero(on.any(1)):
                self.row[i, on[i]] = at
                at += 1
                self.rank_count[d] += 1
        self.rows = at
        v = np.nonzero(valid)
        # of every place in use its entry and its rank's row
        order = np.argsort(self.place[v])
        self.entry = torch.from_numpy((v[0] * K + v[1])[order]).cuda()
        self.row_of = torch.from_numpy(self.row[v][order]).cuda()

    def weights(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn((self.n, self.K), generator=g, device="cuda")

    def at_places(self, seed, more=0, pad=0, scale=1.0):
        """BF16 rows in expert order, NaN behind those in use; pad: elements between rows."""
        t = torch.full((self.places + more, self.H + pad), float("nan"), dtype=BF16, device="cuda")[:, :self.H]
        t[:self.places] = normal((self.places, self.H), seed, scale)
        return t

    def at_rows(self, seed, more=0, pad=0, scale=1.0):
        t = torch.full((self.rows + more, self.H + pad), float("nan"), dtype=BF16, device="cuda")[:, :self.H]
        t[:self.rows] = normal((self.rows, self.H), seed, scale)
        return t

    def stale(self, rows, pad=0):
        return torch.full((rows, self.H + pad), STALE, dtype=BF16, device="cuda")[:, :self.H]

    # References in 64 bits and their bounds
    def unsorted(self, y, w):
        """Sums at the ranks' rows of y (at the places), weighted by w or not, and the bound of an fp32 chain."""
        y = y[:self.places].to(D)
        c = w.reshape(-1)[self.entry].to(D)[:, None] if w is not None else 1.0
        v, m = (torch.zeros((self.rows, self.H), dtype=D, device="cuda") for _ in range(2))
        v.index_add_(0, self.row_of, y * c)
        m.index_add_(0, self.row_of, (y * c).abs())
        return v, self.K * 2.0 ** -24 * m + HALF * 1.01 * v.abs() + 1e-38

    def spread(self, g, w):
        """Gradients at the places of the rows' g."""
        v = g[:self.rows].to(D)[self.row_of] * w.reshape(-1)[self.entry].to(D)[:, None]
        return v, (2.0 ** -24 + HALF * 1.01) * v.abs() + 1e-38

    def dots(self, g, y):
        p = g[:self.rows].to(D)[self.row_of] * y[:self.places].to(D)
        v, m = (torch.zeros(self.n * self.K, dtype=D, device="cuda") for _ in range(2))
        v[self.entry], m[self.entry] = p.sum(1), p.abs().sum(1)
        return v.view(self.n, self.K), (self.H * 2.0 ** -24 * m + 1e-38).view(self.n, self.K)

    def close(self):
        ep.ep_destroy_handle(self.handle)
        ep.ep_destroy_group(self.group)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


__all__ = ["Ranks", "STALE", "BF16", "D", "near", "normal"]
