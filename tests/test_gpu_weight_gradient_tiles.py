"""Gradients of weights in bf16 with many tiles: every tile is taken once, whatever rows the experts hold, and nothing
behind the last one is written.

The XCDs share the tiles by the experts' rows, at whole turns of 32 workgroups.  With nearly all rows on the last expert the
last share begins less than half a turn before the end (2080 of 2072 tiles, were it not cut there).
"""
import numpy as np
import pytest
import torch

from expert_util import BF16, D, HALF, Routing, near, normal, row_tensor
from gpu_util import ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def routing(kind, E, T):
    t = np.arange(T)
    if kind == "spread":
        e = t % E
    elif kind == "halves":      # two experts at the ends
        e = np.where(t % 2 == 0, 0, E - 1)
    elif kind == "steps":       # a few rows everywhere, most on one inside
        e = np.where(t < 3 * E, t % E, E // 2)
    else:
        e = np.full(T, {"first": 0, "last": E - 1, "middle": E // 3}[kind])
    return e.astype(np.int32).reshape(T, 1)


@pytest.mark.parametrize("kind", ["last", "first", "middle", "halves", "spread", "steps"])
@pytest.mark.parametrize("E,H,I", [(259, 512, 1024), (347, 768, 512), (90, 1296, 1000)], ids=str)
def test_every_tile_once(E, H, I, kind):
    T = 12288
    say(f"weight gradients of {E} experts, {I} x {H}, rows: {kind}")
    with Routing("ht", 1, T, E, 1, H, seed=1, topk=routing(kind, E, T), max_tokens_per_rank=T) as r:
        x, dy = row_tensor(r, I, 1), row_tensor(r, H, 2)
        w = normal((E, H, I), 3)
        room = torch.full((E + 1, H, I), -7.25, dtype=BF16, device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, w, dy, grad_w=room[:E])
        assert bool((room[E] == -7.25).all()), "written behind the last expert"
        for e, at in enumerate(r.expert_rows):
            if len(at) == 0:
                assert not bool(room[e].any()), e
                continue
            a, b = dy[at].to(D).t(), x[at].to(D)
            want = a @ b
            # an fp32 sum of the rows' products, rounded to bf16: half a step, and of what the sum is off by
            off = len(at) * 2.0 ** -24 * (a.abs() @ b.abs())
            near(room[e], want, off + HALF * (want.abs() + off), f"expert {e}")


@pytest.mark.parametrize("S,T,E,H,I", [(1, 90, 60, 1024, 768), (3, 40, 40, 1024, 768), (12, 9, 48, 1040, 776), (2, 200, 30, 784, 1288)],
                         ids=str)
def test_slots_of_several_sources(S, T, E, H, I):
    """LL: an expert's rows in one run, in runs that are looked up, and in a list; some experts without a row."""
    say(f"weight gradients of {E} experts, {I} x {H}, {S} sources of {T} tokens")
    with Routing("ll", S, T, E, 2, H, seed=2, skip=(0, E // 2, E - 1)) as r:
        x, dy = row_tensor(r, I, 1), row_tensor(r, H, 2)
        room = torch.full((E + 1, H, I), -7.25, dtype=BF16, device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, normal((E, H, I), 3), dy, grad_w=room[:E])
        assert bool((room[E] == -7.25).all()), "written behind the last expert"
        for e, at in enumerate(r.expert_rows):
            a, b = dy[at].to(D).t(), x[at].to(D)
            want = a @ b
            off = len(at) * 2.0 ** -24 * (a.abs() @ b.abs())
            near(room[e], want, off + HALF * (want.abs() + off), f"expert {e}")
