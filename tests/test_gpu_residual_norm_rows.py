"""ep_residual_norm_backward where a workgroup takes several rows (over 256 of them): every kind of gate with and
without a post norm, one and two pieces a thread (over 8192 columns), and in place.  Bounds: test_gpu_residual_norm."""
import pytest
import torch

import test_gpu_residual_norm as norms
from expert_util import BF16, normal
from gpu_util import ep, need_gpu, say
from test_gpu_residual_norm import group  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


CASES = [(700, 2048, "token", True, BF16, 8), (700, 1040, "token", False, torch.float32, 0),
         (700, 1040, "none", True, torch.float32, 8), (700, 2048, "none", False, BF16, 0),
         (700, 1040, "channel", False, BF16, 16), (2500, 512, "token", True, BF16, 0),
         (9001, 256, "channel", True, torch.float32, 0), (600, 8208, "channel", True, torch.float32, 8),
         (600, 8208, "none", True, BF16, 0), (600, 8208, "token", False, BF16, 0),
         (530, 16384, "token", True, torch.float32, 0), (530, 16384, "channel", True, BF16, 0),
         (530, 16384, "none", False, torch.float32, 0)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("with_res", [True, False], ids=["stream_grad", "no_stream_grad"])
def test_backward_of_many_rows(case, with_res, group):  # noqa: F811
    norms.test_backward(case, with_res, group)


@pytest.mark.parametrize("n,H,gate,post", [(1300, 1040, "channel", True), (1300, 1040, "token", True), (600, 2048, "none", True),
                                           (600, 8208, "channel", True), (600, 8208, "token", False)])
def test_in_place(n, H, gate, post, group):  # noqa: F811
    """grad_residual in grad_out_residual's place, grad_y in y's or grad_out_norm's: the bits of separate outputs, the
    next row's values loaded before a row's results are stored."""
    say(f"residual norm backward in place, {n} x {H}, gate {gate}, post {post}")
    gp = group(H)
    x, y, wn, wp, g = norms.inputs(n, H, gate, post, BF16, 0)
    gr, gn = normal((n, H), 6), normal((n, H), 7)
    work = torch.empty(ep.ep_residual_norm_workspace(gp, n), dtype=torch.uint8, device="cuda")
    first = None
    for place in ("apart", "y", "norm"):
        a, c, d = gr.clone(), gn.clone(), y.clone()
        dres, dy = (torch.empty_like(x), torch.empty_like(x)) if place == "apart" else (a, d if place == "y" else c)
        sums = torch.zeros((3, H), device="cuda")
        dgate = None if g is None else sums[2:3] if gate == "channel" else torch.zeros((n, H), dtype=BF16, device="cuda")
        work.fill_(255)
        ep.ep_residual_norm_backward(gp, d, x, a, c, wn, dres, dy, sums[0], work, w_post=wp, gate=g,
                                     grad_w_post=sums[1] if post else None, grad_gate=dgate, residual_scale=0.5,
                                     block_scale=2.0)
        got = [dres.clone(), dy.clone(), sums.clone()] + ([dgate.clone()] if gate == "token" else [])
        assert all(bool(t.isfinite().all()) for t in got), place
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(first, got)), place
