"""ep_expert_quantize on handles that no dispatch has used: the rows in use follow from the counts alone, so a call
needs nothing that another call on the handle (of another stream, or captured and not yet replayed) has enqueued.

Codes and scales are ep_quantize's on the same rows, bit for bit.
"""
import pytest
import torch

from expert_util import FP8, Routing, row_tensor
from gpu_util import A, ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


GEOMETRIES = [("ht", 2, 40, 6, 640), ("ll", 1, 40, 6, 640), ("ll", 3, 40, 6, 640), ("ll", 9, 30, 9, 256)]


class Rows:
    """A routing's rows, the codes and scales they should get, and outputs that hold 7 and -7.25 where nothing is due."""

    def __init__(self, r, C):
        self.r, self.C = r, C
        self.x = row_tensor(r, C, 2, 3.0)
        used = self.x[~r.unused].contiguous()
        self.q, self.s = torch.empty(used.shape, dtype=FP8, device="cuda"), torch.empty((used.shape[0], C // 128), device="cuda")
        one = ep.ep_create_group(mode="ht", num_nodes=1, ranks_per_node=1, num_experts=1, top_k=1, max_nodes_per_token=0,
                                 hidden=C, max_tokens_per_rank=1, num_src_ranks=1, payload="fp8")
        ep.ep_quantize(one, used, self.q, self.s)
        torch.cuda.synchronize()
        ep.ep_destroy_group(one)

    def outputs(self):
        r = self.r
        return (torch.full((r.rows, self.C), 7, dtype=torch.uint8, device="cuda").view(FP8),
                torch.full((r.rows, self.C // 128), -7.25, device="cuda"))

    def clear(self, out):
        out[0].view(torch.uint8).fill_(7)
        out[1].fill_(-7.25)

    def call(self, out):
        ep.ep_expert_quantize(self.r.handle, self.x, *out)

    def check(self, out, what):
        q, s, unused = out[0].view(torch.uint8), out[1], self.r.unused
        assert torch.equal(q[~unused], self.q.view(torch.uint8)) and torch.equal(s[~unused], self.s), what
        assert bool((q[unused] == 7).all()) and bool((s[unused] == -7.25).all()), what


def without_maps(r):
    """The routing's handle made anew where a handle of another routing has left its maps."""
    ep.ep_destroy_handle(r.handle)
    other = ep.ep_create_handle(r.group, r.idx.flip(1).roll(1, 0).contiguous())
    ep.ep_handle_get_map(other, A.EP_MAP_HT_ROW if r.mode == "ht" else A.EP_MAP_LL_SLOT)
    torch.cuda.synchronize()
    ep.ep_destroy_handle(other)
    r.handle = ep.ep_create_handle(r.group, r.idx)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mode,S,T,E,C", GEOMETRIES)
def test_captured_first_and_called_before_the_replay(mode, S, T, E, C):
    say(f"quantise captured first, {mode} {S} x {T}, {E} experts")
    with Routing(mode, S, T, E, 2, 256, seed=9) as r:
        rows = Rows(r, C)
        without_maps(r)
        inside, eager = rows.outputs(), rows.outputs()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rows.call(inside)
        rows.call(eager)
        torch.cuda.synchronize()
        rows.check(eager, "before the replay")
        for turn in range(3):
            rows.clear(inside)
            graph.replay()
            torch.cuda.synchronize()
            rows.check(inside, f"replay {turn}")
            rows.clear(eager)
            rows.call(eager)
            torch.cuda.synchronize()
            rows.check(eager, f"after replay {turn}")


@pytest.mark.parametrize("mode,S,T,E,C", GEOMETRIES)
def test_second_stream_does_not_wait_for_the_first(mode, S, T, E, C):
    say(f"quantise on two streams, {mode} {S} x {T}, {E} experts")
    with Routing(mode, S, T, E, 2, 256, seed=9) as r:
        rows = Rows(r, C)
        without_maps(r)
        late, early = rows.outputs(), rows.outputs()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            torch.cuda._sleep(20_000_000)
            rows.call(late)
        with torch.cuda.stream(b):
            rows.call(early)
        b.synchronize()
        rows.check(early, "second stream")
        a.synchronize()
        rows.check(late, "first stream")


@pytest.mark.parametrize("mode,S,T,E,K,C", [("ll", 64, 2, 128, 3, 256), ("ll", 1, 300, 2, 2, 8320), ("ht", 1, 300, 3, 2, 8320),
                                            ("ht", 1, 700, 80, 4, 128), ("ll", 1, 5, 64, 1, 4224)])
def test_many_counts_and_wide_rows(mode, S, T, E, K, C):
    """More counts than workgroups are spread over, rows of several waves, most counts zero."""
    say(f"quantise, {mode} {S} x {T}, {E} experts, {C} columns")
    with Routing(mode, S, T, E, K, 256, seed=4) as r:
        rows = Rows(r, C)
        out = rows.outputs()
        rows.call(out)
        torch.cuda.synchronize()
        rows.check(out, "rows")
        assert ep.ep_get_device_error(r.group) == 0
