"""The experts' products in captured graphs: all of them in one graph, two graphs of one handle on two streams at
once, replayed with new inputs and the program's own eager calls between.  Every replay has the eager calls' bits.
"""
import pytest
import torch

from expert_util import BF16, FP8, Routing, gated, near, normal, out_tensor, product, row_tensor
from gpu_util import A, ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Step:
    """Every product of the block, forward and backward, between buffers of its own."""

    def __init__(self, r, I, seed):
        E, H = r.E, r.H
        self.r, self.I = r, I
        self.x = row_tensor(r, H, seed)
        self.g = row_tensor(r, H, seed + 1)
        self.wg, self.wu = (normal((E, I, H), seed + i, H ** -0.5) for i in (2, 3))
        self.wd = normal((E, H, I), seed + 4, I ** -0.5)
        self.qd = (self.wd / 0.01).clamp(-448, 448).to(FP8)
        self.sd = torch.full((E, (H + 127) // 128, I // 128), 0.01, device="cuda")
        self.fresh()

    def fresh(self):
        r, E, H, I = self.r, self.r.E, self.r.H, self.I
        self.a, self.da, self.dg, self.du = (out_tensor(r, I) for _ in range(4))
        self.y, self.y8, self.dx = (out_tensor(r, H) for _ in range(3))
        self.q = torch.zeros((r.rows, I), dtype=torch.uint8, device="cuda").view(FP8)
        self.qs = torch.zeros((r.rows, I // 128), device="cuda")
        self.dwg, self.dwu = (torch.zeros((E, I, H), dtype=BF16, device="cuda") for _ in range(2))
        self.dwd = torch.zeros((E, H, I), device="cuda")

    def run(self):
        h = self.r.handle
        ep.ep_expert_gated(h, self.x, self.wg, self.wu, self.a)
        ep.ep_expert_linear(h, self.a, self.wd, self.y)
        ep.ep_expert_quantize(h, self.a, self.q, self.qs)
        ep.ep_expert_linear(h, self.q, self.qd, self.y8, x_scales=self.qs, w_scales=self.sd)
        ep.ep_expert_linear_backward(h, self.a, self.wd, self.g, grad_x=self.da, grad_w=self.dwd)
        ep.ep_expert_gated_backward(h, self.x, self.wg, self.wu, self.da, self.dg, self.du, grad_rows=self.dx,
                                    grad_w_gate=self.dwg, grad_w_up=self.dwu)

    def results(self):
        return [t.clone() for t in (self.a, self.y, self.q.view(torch.uint8), self.qs, self.y8, self.da, self.dg, self.du,
                                    self.dx, self.dwg, self.dwu, self.dwd)]

    def load(self, seed):
        self.x.copy_(row_tensor(self.r, self.r.H, seed))
        self.g.copy_(row_tensor(self.r, self.r.H, seed + 50))


@pytest.mark.parametrize("mode,S,T,E", [("ht", 1, 90, 6), ("ll", 3, 40, 6), ("ll", 9, 30, 9), ("ll", 2, 60, 80)])
def test_two_graphs_of_one_handle(mode, S, T, E):
    say(f"two graphs of one handle, {mode} {S} x {T}, {E} experts")
    K, H, I = 2, 384, 256
    with Routing(mode, S, T, E, K, H, seed=3) as r:
        if mode == "ht":   # the row map: written by a dispatch, or here
            ep.ep_handle_get_map(r.handle, A.EP_MAP_HT_ROW)
        else:
            ep.ep_handle_get_map(r.handle, A.EP_MAP_LL_SLOT)
        steps = [Step(r, I, 10), Step(r, I, 30)]
        graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
        for st in steps:
            st.run()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                st.run()
            graphs.append(g)
        for turn in range(3):
            want = []
            for i, st in enumerate(steps):
                st.load(100 * turn + i)
                st.run()
                want.append(st.results())
                for t in (st.a, st.y, st.y8, st.da, st.dg, st.du, st.dx):
                    t[~r.unused] = -7.25
                for t in (st.q.view(torch.uint8), st.qs, st.dwg, st.dwu, st.dwd):
                    t.zero_()
            torch.cuda.synchronize()
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for st, w in zip(steps, want):
                for k, (a, b) in enumerate(zip(w, st.results())):
                    assert torch.equal(a.nan_to_num(9.0) if a.is_floating_point() else a,
                                       b.nan_to_num(9.0) if b.is_floating_point() else b), (turn, k)
        assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("mode,S", [("ht", 1), ("ll", 3), ("ll", 9)])
def test_every_entry_names_one_expert(mode, S):
    """All tokens name one expert in all their entries: it holds each token once, the others nothing."""
    say(f"one expert for everything, {mode} {S}")
    T, E, K, H, I = 270 // S, 9, 3, 256, 128
    topk = torch.full((S * T, K), 4, dtype=torch.int32).numpy()
    with Routing(mode, S, T, E, K, H, topk=topk) as r:
        assert len(r.expert_rows[4]) == S * T
        st = Step(r, I, 5)
        st.run()
        x = st.x[r.expert_rows[4]].double()
        near(st.a[r.expert_rows[4]], *gated(product(x, st.wg[4].double()), product(x, st.wu[4].double()), "silu"))
        near(st.dwd[4], *product(st.g[r.expert_rows[4]].double().t(), st.a[r.expert_rows[4]].double().t()))
        others = [e for e in range(E) if e != 4]
        assert not bool(st.dwd[others].any()) and not bool(st.dwg[others].any()) and not bool(st.dwu[others].any())
        assert bool((st.a[r.unused] == -7.25).all()) and bool((st.dx[r.unused] == -7.25).all())
