"""Inputs, routings and 64-bit references of the experts' products (not collected by pytest).

Error bounds, per element, used by the tests:
  * an fp32 sum of K products in any order is within K 2^-24 sum|a b| of the exact one
    (K roundings of partial sums, each at most half a step of at most sum|a b|);
  * a rounding to bf16 is off by at most 2^-8 of the value;
  * one E4M3 matrix instruction aligns its 128 products to the largest: 2.4e-4 (2^-12) of the
    largest product is the worst of 4096 such sums over all code pairs, 2^-11 is allowed;
  * the activations use exp and reciprocal instructions: within 2^-18 of the value for |g| < 32
    (an argument error of |g| 2^-23 and a few steps of 2^-23).
"""
from __future__ import annotations

import numpy as np
import torch

from gpu_util import A, ep

D = torch.float64
BF16 = torch.bfloat16
FP8 = torch.float8_e4m3fn
HALF = 2.0 ** -8


class Routing:
    """A group, a handle and the rows its experts hold, worked out on the host."""

    def __init__(self, mode="ht", S=1, T=8, E=8, K=2, H=256, payload="bf16", seed=0, skip=(), topk=None, **over):
        rng = np.random.default_rng(seed)
        self.n = n = S * T
        if topk is None:
            score = rng.random((n, E))
            if n >= 2000:
                score += np.linspace(0, 0.8, E)   # a handful to several hundred rows an expert
            score[:, list(skip)] = -1.0           # experts that receive nothing
            topk = np.argsort(-score, axis=1)[:, :K].astype(np.int32)
        self.topk = topk
        self.E, self.S, self.T, self.K, self.H, self.mode = E, S, T, K, H, mode
        ranks = max(r for r in (1, 2, 4, 8, 16) if E % r == 0)
        nodes = 2 if S > ranks and E % (2 * ranks) == 0 else 1
        ranks = E if S > nodes * ranks else ranks
        nodes = 1 if ranks == E else nodes
        cfg = dict(mode=mode, num_nodes=nodes, ranks_per_node=ranks, num_experts=E, top_k=K, max_nodes_per_token=0,
                   hidden=H, max_tokens_per_rank=T, num_src_ranks=S, payload=payload)
        cfg.update(over)
        self.slots = cfg["max_tokens_per_rank"]
        self.group = ep.ep_create_group(**cfg)
        self.idx = torch.from_numpy(topk).cuda()
        self.handle = ep.ep_create_handle(self.group, self.idx)
        rows = [[] for _ in range(E)]
        where = {}
        if mode == "ht":
            per = [[] for _ in range(E)]
            for i in range(n):
                for k in range(K):
                    e = topk[i, k]
                    if 0 <= e < E and e not in topk[i, :k]:
                        per[e].append((i, k))
            at = 0
            for e in range(E):
                for i, k in per[e]:
                    rows[e].append(at)
                    where[(i, k)] = at
                    at += 1
            self.rows = max(at, 1)
        else:
            used = np.zeros((E, S), np.int64)
            for i in range(n):
                for k in range(K):
                    e = topk[i, k]
                    if 0 <= e < E and e not in topk[i, :k]:
                        s = i // T
                        where[(i, k)] = (e * S + s) * self.slots + used[e, s]
                        used[e, s] += 1
            for e in range(E):
                for s in range(S):
                    rows[e] += [(e * S + s) * self.slots + j for j in range(used[e, s])]
            self.rows = E * S * self.slots
        self.expert_rows = [torch.tensor(r, dtype=torch.int64, device="cuda") for r in rows]
        self.where = where
        used = torch.zeros(self.rows, dtype=torch.bool)
        for r in rows:
            used[r] = True
        self.unused = (~used).cuda()

    def close(self):
        ep.ep_destroy_handle(self.handle)
        ep.ep_destroy_group(self.group)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()


def normal(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def row_tensor(r: Routing, cols, seed, scale=1.0, pad=0, stale=float("nan")):
    """BF16 [rows, cols] with NaN in the rows that hold nothing; pad: extra elements per row."""
    t = torch.full((r.rows, cols + pad), stale, dtype=BF16, device="cuda")[:, :cols]
    t[~r.unused] = normal((int((~r.unused).sum()), cols), seed, scale)
    return t


def out_tensor(r: Routing, cols, pad=0, dtype=BF16):
    return torch.full((r.rows, cols + pad), -7.25, dtype=dtype, device="cuda")[:, :cols]


def untouched(r: Routing, t):
    assert bool((t[r.unused] == -7.25).all()), "a row that holds nothing was written"


def near(got, want, bound, what=""):
    got = got.to(D)
    bad = ~((got - want).abs() <= bound)
    if bool(bad.any()):
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got.reshape(-1)[i].item()} for {want.reshape(-1)[i].item()} "
                             f"+- {bound.reshape(-1)[i].item()}")


def act64(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = (8 / torch.pi) ** 0.5
    s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def product(a, b):
    """a b^T in 64 bits and the bound on an fp32 evaluation of it."""
    return a @ b.t(), a.shape[1] * 2.0 ** -24 * (a.abs() @ b.abs().t())


def product_fp8(qa, sa, qb, sb):
    """The same for codes and scales (qa [R, C], sa [R, C/128], qb [N, C], sb [N/128 up, C/128])."""
    R, C = qa.shape
    N = qb.shape[0]
    y = torch.zeros((R, N), dtype=D, device=qa.device)
    b = torch.zeros_like(y)
    mag = torch.zeros_like(y)
    for c in range(C // 128):
        x = qa[:, c * 128:(c + 1) * 128].to(D)
        w = qb[:, c * 128:(c + 1) * 128].to(D)
        s = sa[:, c, None].to(D) * sb[:, c].to(D).repeat_interleave(128)[None, :N]
        y += (x @ w.t()) * s
        mag += (x.abs() @ w.abs().t()) * s
        # the largest product is at most (largest |x|) (largest |w|)
        b += 2.0 ** -11 * x.abs().amax(1)[:, None] * w.abs().amax(1)[None, :] * s
    return y, b + (C // 128 + 2) * 2.0 ** -23 * mag


def gated(pre, up, kind):
    """Value and bound of act(g) u from (g, bound), (u, bound)."""
    (g, bg), (u, bu) = pre, up
    f, df = act64(g, kind)
    v = f * u
    # |act'| <= 1.13 for both; second-order terms of the small bounds are covered by the factor
    b = 1.2 * bg * (u.abs() + bu) + f.abs() * bu + (2.0 ** -18 + HALF) * v.abs() * 1.01
    return v, b + 1e-30
