"""The experts' products at the limits of a routing and of its tensors: as many experts as a group takes (up to 16 a
lane in the scan), 32 entries a token, tensors of more rows than are in use with NaN behind them, more slots than
tokens, every 3-D form, gradients of weights with strides.  Bounds: see expert_util."""
import pytest
import torch

from expert_util import BF16, D, FP8, HALF, Routing, gated, near, normal, out_tensor, product, product_fp8, row_tensor, \
    untouched
from gpu_util import A, ep, need_gpu, say
from test_gpu_experts import check_weight_grad, weights, weights_fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def check_all(r, H, I, x, dy):
    """Gated and linear products and both backward passes of a routing."""
    E = r.E
    wg, wu, wd = weights(E, I, H, 3), weights(E, I, H, 4), weights(E, H, I, 5)
    a, y, da, dg, du, dx = (out_tensor(r, c) for c in (I, H, I, I, I, H))
    dwg, dwu = (torch.full((E, I, H), 9.0, device="cuda") for _ in range(2))
    dwd = torch.full((E, H, I), 9.0, dtype=BF16, device="cuda")
    ep.ep_expert_gated(r.handle, x, wg, wu, a)
    ep.ep_expert_linear(r.handle, a, wd, y)
    ep.ep_expert_linear_backward(r.handle, a, wd, dy, grad_x=da, grad_w=dwd)
    ep.ep_expert_gated_backward(r.handle, x, wg, wu, da, dg, du, grad_rows=dx, grad_w_gate=dwg, grad_w_up=dwu)
    for e, at in enumerate(r.expert_rows):
        if len(at):
            xe = x[at].to(D)
            near(a[at], *gated(product(xe, wg[e].to(D)), product(xe, wu[e].to(D)), "silu"), f"gated {e}")
            v, b = product(a[at].to(D), wd[e].to(D))
            near(y[at], v, b + HALF * v.abs() * 1.01, f"linear {e}")
            v, b = product(dy[at].to(D), wd[e].to(D).t())
            near(da[at], v, b + HALF * v.abs() * 1.01, f"gradient of the linear product's rows {e}")
            (p, bp), (q, bq) = product(dg[at].to(D), wg[e].to(D).t()), product(du[at].to(D), wu[e].to(D).t())
            near(dx[at], p + q, 2 * (bp + bq) + HALF * (p + q).abs() * 1.01, f"gradient of the rows {e}")
    check_weight_grad(r, dwd, dy, a, "linear")
    check_weight_grad(r, dwg, dg, x, "gate")
    check_weight_grad(r, dwu, du, x, "up")
    for t in (a, y, da, dg, du, dx):
        untouched(r, t)
    assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("mode,S,T,E,K", [("ht", 1, 70, 1024, 8), ("ll", 1, 40, 1024, 8), ("ll", 2, 20, 1024, 32),
                                          ("ht", 2, 9, 1000, 32), ("ll", 1, 33, 80, 2), ("ll", 2, 17, 65, 3)])
def test_many_experts(mode, S, T, E, K):
    say(f"products of {E} experts, {mode} {S} x {T}, top-{K}")
    H, I = 64, 40
    over = dict(num_nodes=1, ranks_per_node=E) if E == 65 else {}
    with Routing(mode, S, T, E, K, H, seed=2, **over) as r:
        check_all(r, H, I, row_tensor(r, H, 6), row_tensor(r, H, 7))


@pytest.mark.parametrize("mode,S,T,slots", [("ht", 2, 50, 90), ("ll", 1, 50, 90), ("ll", 3, 20, 64), ("ll", 12, 9, 11)])
def test_more_rows_than_in_use(mode, S, T, slots):
    """A group for more tokens than the batch has; in HT also tensors of all its rows, NaN behind the ones in use."""
    say(f"products in larger tensors, {mode} {S} x {T} of {slots}")
    E, K, H, I = 12, 3, 144, 72
    with Routing(mode, S, T, E, K, H, seed=3, max_tokens_per_rank=slots) as r:
        if mode == "ht":
            used = r.rows
            r.rows = S * slots * K
            r.unused = torch.arange(r.rows, device="cuda") >= used
        check_all(r, H, I, row_tensor(r, H, 6), row_tensor(r, H, 7))


@pytest.mark.parametrize("S", [1, 3, 12])
def test_three_dimensions(S):
    """LL tensors as [E, S*T_max, C]: the same bits as [rows, C]."""
    say(f"products on 3-D tensors, {S} sources")
    E, H, I, T = 12, 256, 128, 10
    with Routing("ll", S, T, E, 2, H, seed=4) as r:
        x = row_tensor(r, H, 1)
        wg, wu, wd = weights(E, I, H, 2), weights(E, I, H, 3), weights(E, H, I, 4)
        q8, s8 = weights_fp8(E, H, I, 5)
        got = []
        for shape in ((lambda c: (r.rows, c)), (lambda c: (E, S * T, c))):
            new = lambda c, t=BF16: torch.zeros(shape(c), dtype=t, device="cuda")
            a, y, y8, da, dg, du, dx, s = new(I), new(H), new(H), new(I), new(I), new(I), new(H), new(1, torch.float32)
            q = new(I, torch.uint8).view(FP8)
            dwd, dwg, dwu = (torch.zeros(w.shape, device="cuda") for w in (wd, wg, wu))
            xv = x.view(shape(H))
            ep.ep_expert_gated(r.handle, xv, wg, wu, a)
            ep.ep_expert_linear(r.handle, a, wd, y)
            ep.ep_expert_quantize(r.handle, a, q, s)
            ep.ep_expert_linear(r.handle, q, q8, y8, x_scales=s, w_scales=s8)
            ep.ep_expert_linear_backward(r.handle, a, wd, xv, grad_x=da, grad_w=dwd)
            ep.ep_expert_gated_backward(r.handle, xv, wg, wu, da, dg, du, grad_rows=dx, grad_w_gate=dwg, grad_w_up=dwu)
            flat = [t.reshape(r.rows, -1) for t in (a, y, y8, da, dg, du, dx, s, q.view(torch.uint8))]
            got.append(flat + [dwd, dwg, dwu])
        for k, (p, w) in enumerate(zip(*got)):
            assert torch.equal(p, w), k
        for e, at in enumerate(r.expert_rows):
            if len(at):
                v, b = product_fp8(got[0][8][at].view(FP8), got[0][7][at], q8[e], s8[e])
                near(got[0][2][at], v, b + HALF * v.abs() * 1.01, f"expert {e}")


@pytest.mark.parametrize("wtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [40, 900])
def test_weight_gradients_with_strides(wtype, T):
    """Matrices and rows further apart than they are long: what lies between keeps its values."""
    say(f"weight gradients with strides, {T} tokens, {wtype}")
    E, H, I = 10, 272, 264
    with Routing("ht", 1, T, E, 2, H, seed=5) as r:
        x, dy, w = row_tensor(r, I, 1), row_tensor(r, H, 2), weights(E, H, I, 3)
        big = torch.full((E, H + 3, I + 16), 9.0, dtype=wtype, device="cuda")
        dw = big[:, :H, :I]
        ep.ep_expert_linear_backward(r.handle, x, w, dy, grad_w=dw)
        check_weight_grad(r, dw, dy, x, "weights")
        assert bool((big[:, H:] == 9.0).all()) and bool((big[:, :, I:] == 9.0).all())
