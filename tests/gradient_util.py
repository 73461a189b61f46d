"""Gradients against differences of a 64-bit loss (not collected by pytest).

A gradient `got` is compared one tensor at a time, along directions of norm about 1 in which a mistake shows:
  * along `got` itself: v = got/|got| + r/8, r a random vector of norm 1;
  * along what `got` differs in from `ref`, the formula's gradient in 64 bits: v = (got - ref)/|got - ref|.
If got = g + d with the true gradient g and |d| <= delta |g|, then |<got, v> - <g, v>| <= delta |g||v|.  Along `got` a
flipped sign gives 2 |g||v| nearly, and this check does not need `ref` to be right; along got - ref, with ref = g, the
left side is |d| itself, whatever part of the gradient is wrong or missing.  A random direction in N dimensions would
see |d|/sqrt(N) of either, less than the bound.

A central difference of step h around a point adds the loss's own rounding (2^-53 of its terms over h) and h^2 of its
third derivative, both far below delta here.
"""
from __future__ import annotations

import torch

D = torch.float64


def directions(got, ref):
    got, ref = got.to(D), ref.to(D)
    for seed in range(2):
        r = torch.randn(got.shape, generator=torch.Generator().manual_seed(seed), dtype=D).to(got.device)
        yield got / got.norm() + r / (8 * r.norm())
    off = got - ref
    if float(off.norm()) > 0:
        yield off / off.norm()


def difference(loss, point, v, step=1e-5):
    """d loss(point + t v) / dt at 0."""
    return (float(loss(point + step * v)) - float(loss(point - step * v))) / (2 * step)


def mismatch(got, ref, loss, point, delta):
    """The first direction along which the gradient `got` of `loss` at `point` is further than delta of itself from
    the difference: (its number, both sides, the bound); None if there is none."""
    for k, v in enumerate(directions(got, ref)):
        ours, theirs = float((got.to(D) * v).sum()), difference(loss, point, v)
        bound = delta * float(got.to(D).norm() * v.norm())
        if not abs(ours - theirs) <= bound:
            return k, ours, theirs, bound
    return None


def check(got, ref, loss, point, delta, what):
    assert bool(torch.isfinite(got).all()) and float(got.to(D).norm()) > 0, what
    bad = mismatch(got, ref, loss, point, delta)
    assert bad is None, (what, *bad)
