"""The maps of a handle that no dispatch has used, first asked for by a captured call: the graph holds the pass that
writes them, so a call outside of it writes them itself and does not read what no replay has written yet."""
import pytest
import torch

from expert_util import Routing, normal, row_tensor
from gpu_util import A, ep, need_gpu, say
from test_gpu_experts_quantize import without_maps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


E, K, H = 6, 2, 256


class Calls:
    """What needs the maps, into outputs of its own."""

    def __init__(self, r, y, up, tw):
        self.r, self.y, self.up, self.tw = r, y, up, tw
        self.tokens = torch.zeros_like(up)
        self.rows, self.weights = torch.zeros_like(y), torch.zeros_like(tw)

    def run(self, what):
        h = self.r.handle
        if what == "combine":
            ep.ep_combine(h, self.y, self.tw, self.tokens)
        elif what == "combine_backward":
            ep.ep_combine_backward(h, self.up, self.tw, self.rows, expert_out=self.y, grad_weights=self.weights)
        else:
            ep.ep_dispatch_backward(h, self.y, self.tokens)

    def take(self):
        torch.cuda.synchronize()
        got = [t.clone() for t in (self.tokens, self.rows, self.weights)]
        for t in (self.tokens, self.rows, self.weights):
            t.zero_()
        torch.cuda.synchronize()
        return got


@pytest.mark.parametrize("what", ["combine", "combine_backward", "dispatch_backward"])
@pytest.mark.parametrize("mode,S,T", [("ht", 2, 50), ("ll", 3, 40)])
def test_captured_first_and_called_before_the_replay(mode, S, T, what):
    say(f"{what} captured first, {mode} {S} x {T}")
    with Routing(mode, S, T, E, K, H, seed=5) as r, Routing(mode, S, T, E, K, H, seed=5) as ready:
        ep.ep_handle_get_map(ready.handle, A.EP_MAP_HT_ROW if mode == "ht" else A.EP_MAP_LL_SLOT)
        data = row_tensor(r, H, 1, stale=0.0), normal((S * T, H), 2), torch.softmax(normal((S * T, K), 3).float(), 1)
        want = Calls(ready, *data)
        want.run(what)
        want = want.take()
        assert any(bool(t.any()) for t in want)

        without_maps(r)
        inside, eager = Calls(r, *data), Calls(r, *data)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            inside.run(what)
            inside.run(what)
        eager.run(what)
        assert all(torch.equal(a, b) for a, b in zip(eager.take(), want)), "before the replay"
        for turn in range(3):
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(inside.take(), want)), f"replay {turn}"
            eager.run(what)
            assert all(torch.equal(a, b) for a, b in zip(eager.take(), want)), f"after replay {turn}"
        got = ep.ep_handle_get_map(r.handle, A.EP_MAP_HT_ROW if mode == "ht" else A.EP_MAP_LL_SLOT).cpu()
        assert all(int(got[i, k]) == row for (i, k), row in r.where.items())
