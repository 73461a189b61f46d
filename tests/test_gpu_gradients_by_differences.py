"""The experts' products' and the norms' backward passes against differences of their 64-bit formulas, one gradient at
a time, along directions in which a mistake shows (see gradient_util; its CPU test says what is noticed).

Bounds.  The kernels' gradient is g + d with |d| <= b element by element, so that a difference along v is met within
|b||v|: `delta` is |b|/|g|.  For the products
  * grad_gate and grad_up, rounded to bf16 (2^-8 of the value) from activations within 2^-18 and fp32 sums of up to 64
    products (2^-18 of the magnitudes), are within e = 2^-8 1.05 |value| + 2^-14 |dA| (|u| or |g|);
  * what is summed from them is within the same sum of e and magnitudes, a bf16 result 2^-8 of itself further;
  * the linear product's gradients are sums of K exact products: K 2^-24 of the magnitudes, and 2^-8 if rounded.
"""
import pytest
import torch

import test_gpu_residual_norm as norms
from expert_util import BF16, D, HALF, Routing, act64, normal, out_tensor, row_tensor
from gradient_util import check
from gpu_util import A, ep, need_gpu, say
from test_gpu_experts_calls import block_reference, weights
from test_gpu_residual_norm import group  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def delta(b, g):
    return float(b.norm() / g.norm()) + 2.0 ** -30


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("mode,S,T,grad", [("ht", 1, 9, "f32"), ("ht", 1, 150, "bf16"), ("ll", 3, 20, "f32")])
def test_gated(mode, S, T, grad, act):
    say(f"gated gradients by differences, {mode} {S} x {T}, {act}, {grad}")
    E, H, I = 3, 64, 40
    gtype = torch.float32 if grad == "f32" else BF16
    with Routing(mode, S, T, E, 2, H, seed=13) as r:
        x, da = row_tensor(r, H, 1), row_tensor(r, I, 4)
        wg, wu = weights(E, I, H, 2), weights(E, I, H, 3)
        dg, du, dx = out_tensor(r, I), out_tensor(r, I), out_tensor(r, H)
        d1, d2 = torch.empty((E, I, H), dtype=gtype, device="cuda"), torch.empty((E, I, H), dtype=gtype, device="cuda")
        ep.ep_expert_gated_backward(r.handle, x, wg, wu, da, dg, du, activation=act, grad_rows=dx, grad_w_gate=d1,
                                    grad_w_up=d2)
        used = torch.cat(r.expert_rows)
        X, DA, WG, WU = x[used].to(D), da[used].to(D), wg.to(D), wu.to(D)
        n = [len(t) for t in r.expert_rows]

        def loss(X, WG, WU):
            total = 0.0
            for e, (xe, de) in enumerate(zip(X.split(n), DA.split(n))):
                f, _ = act64(xe @ WG[e].t(), act)
                total += float((f * (xe @ WU[e].t()) * de).sum())
            return total
        ref, bound = [[], [], []], [[], [], []]
        for e, (xe, de) in enumerate(zip(X.split(n), DA.split(n))):
            g, u = xe @ WG[e].t(), xe @ WU[e].t()
            f, df = act64(g, act)
            pg, pu = de * u * df, de * f
            eg = 1.05 * HALF * pg.abs() + 2.0 ** -14 * (de * u).abs()
            eu = 1.05 * HALF * pu.abs() + 2.0 ** -14 * (de * g).abs()
            for k, (v, b) in enumerate(((pg @ WG[e] + pu @ WU[e], eg @ WG[e].abs() + eu @ WU[e].abs()),
                                        (pg.t() @ xe, eg.t() @ xe.abs()), (pu.t() @ xe, eu.t() @ xe.abs()))):
                ref[k].append(v)
                bound[k].append(b + (1.05 * HALF * v.abs() if k == 0 or grad == "bf16" else 0))
        ref = [torch.cat(ref[0]), torch.stack(ref[1]), torch.stack(ref[2])]
        bound = [torch.cat(bound[0]), torch.stack(bound[1]), torch.stack(bound[2])]
        for k, (got, what) in enumerate(((dx[used], "rows"), (d1, "gate"), (d2, "up"))):
            point = [X, WG, WU]
            check(got, ref[k], lambda t: loss(*point[:k], t, *point[k + 1:]), point[k], delta(bound[k], ref[k]), what)


@pytest.mark.parametrize("mode,S,T,grad", [("ht", 1, 9, "f32"), ("ht", 1, 150, "bf16"), ("ll", 3, 20, "f32")])
def test_linear(mode, S, T, grad):
    say(f"linear gradients by differences, {mode} {S} x {T}, {grad}")
    E, N, C = 3, 64, 40
    gtype = torch.float32 if grad == "f32" else BF16
    with Routing(mode, S, T, E, 2, 64, seed=17) as r:
        x, dy, w = row_tensor(r, C, 1), row_tensor(r, N, 2), weights(E, N, C, 3)
        dx, dw = out_tensor(r, C), torch.empty((E, N, C), dtype=gtype, device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, w, dy, grad_x=dx, grad_w=dw)
        used = torch.cat(r.expert_rows)
        X, DY, W = x[used].to(D), dy[used].to(D), w.to(D)
        n = [len(t) for t in r.expert_rows]

        def loss(X, W):
            return sum(float(((xe @ W[e].t()) * de).sum()) for e, (xe, de) in enumerate(zip(X.split(n), DY.split(n))))
        parts = list(zip(X.split(n), DY.split(n)))
        rx = torch.cat([de @ W[e] for e, (_, de) in enumerate(parts)])
        bx = torch.cat([N * 2.0 ** -24 * (de.abs() @ W[e].abs()) for e, (_, de) in enumerate(parts)]) + 1.05 * HALF * rx.abs()
        rw = torch.stack([de.t() @ xe for xe, de in parts])
        bw = torch.stack([len(xe) * 2.0 ** -24 * (de.abs().t() @ xe.abs()) for xe, de in parts])
        bw = bw + (1.05 * HALF * rw.abs() if grad == "bf16" else 0)
        check(dx[used], rx, lambda t: loss(t, W), X, delta(bx, rx), "rows")
        check(dw, rw, lambda t: loss(X, t), W, delta(bw, rw), "weights")


@pytest.mark.parametrize("n,H,gate,post", [(5, 64, "channel", True), (300, 48, "token", True), (700, 64, "channel", False),
                                           (3, 272, "none", True), (600, 32, "token", False)])
def test_norms(n, H, gate, post, group):  # noqa: F811
    """The stream is given to the backward pass: the residual is what makes it so, in 64 bits.  Bounds: those of
    test_gpu_residual_norm."""
    say(f"norm gradients by differences, {n} x {H}, gate {gate}, post {post}")
    x, y, wn, wp, g = norms.inputs(n, H, gate, post, torch.float32, 0)
    a, b, eps = 0.5, -0.75, 1e-5
    gr, gn = normal((n, H), 6), normal((n, H), 7)
    dres, dy = torch.empty((n, H), dtype=BF16, device="cuda"), torch.empty((n, H), dtype=BF16, device="cuda")
    sums = torch.empty((3, H), device="cuda")
    dgate = None if g is None else sums[2:3] if gate == "channel" else torch.empty((n, H), dtype=BF16, device="cuda")
    gp = group(H)
    work = torch.empty(ep.ep_residual_norm_workspace(gp, n), dtype=torch.uint8, device="cuda")
    ep.ep_residual_norm_backward(gp, y, x, gr, gn, wn, dres, dy, sums[0], work, w_post=wp, gate=g,
                                 grad_w_post=sums[1] if post else None, grad_gate=dgate, residual_scale=a, block_scale=b,
                                 eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))

    def branch(y, wp, g):
        t = y * norms.rms(y, eps) * wp if post else y
        return b * (t if g is None else t * g)

    def forward(res, y, wn, wp, g):
        stream = a * res + branch(y, wp, g)
        return (stream * gr.to(D)).sum() + (stream * norms.rms(stream, eps) * wn * gn.to(D)).sum()
    Y, WN = y.to(D), wn.to(D)
    WP, G = wp.to(D) if post else None, None if g is None else g.to(D)
    point = [(x.to(D) - branch(Y, WP, G)) / a, Y, WN, WP, G]
    leaves = [None if t is None else t.clone().requires_grad_() for t in point]
    forward(*leaves).backward()
    slack = (H + n + 32) * 2.0 ** -23 * 1.1
    X, r = x.to(D), norms.rms(x.to(D), eps)
    vm = (gn.to(D) * WN).abs()
    mag = gr.to(D).abs() + r * (vm + (X * r).abs() * (vm * (X * r).abs()).mean(1, keepdim=True))
    ry = norms.rms(Y, eps) if post else torch.ones((n, 1), dtype=D, device="cuda")
    wpm = WP.abs() if post else 1
    dtm = abs(b) * mag * (1 if G is None else G.abs())
    ym = dtm
    if post:
        ym = ry * (dtm * wpm + (Y * ry).abs() * (dtm * wpm * (Y * ry).abs()).mean(1, keepdim=True))
    tm = (Y * ry).abs() * wpm
    rounded = lambda t: 1.01 * HALF * t.grad.abs()
    todo = [(0, dres, slack * abs(a) * mag + rounded(leaves[0]), "residual"), (1, dy, slack * ym + rounded(leaves[1]), "y"),
            (2, sums[0], slack * (gn.to(D) * X * r).abs().sum(0), "w_pre")]
    if post:
        todo.append((3, sums[1], slack * (dtm * (Y * ry).abs()).sum(0), "w_post"))
    if gate == "channel":
        todo.append((4, dgate, slack * (abs(b) * mag * tm).sum(0, keepdim=True), "gate"))
    elif gate == "token":
        todo.append((4, dgate, slack * abs(b) * mag * tm + rounded(leaves[4]), "gate"))
    for k, got, bound, what in todo:
        check(got, leaves[k].grad, lambda t: forward(*point[:k], t, *point[k + 1:]), point[k], delta(bound, leaves[k].grad),
              what)


@pytest.mark.parametrize("mode", ["ht", "ll"])
def test_block(mode):
    """Norm, dispatch, experts, weighted combine and residual: the chain's backward calls, every gradient against
    differences of the 64-bit block.  Up to 10 bf16 tensors lie on the longest path, each off by 2^-8 of itself at
    most, errors of random sign: 10 2^-8 of a gradient's norm."""
    say(f"gradients of the block by differences, {mode}")
    E, K, H, I, S, T = 8, 2, 256, 128, 2, 12
    n = S * T
    with Routing(mode, S, T, E, K, H, seed=11) as r:
        h, g = r.handle, r.group
        x, up = normal((n, H), 1), normal((n, H), 7)
        wn = 1 + normal((H,), 2, 0.1, torch.float32)
        wg, wu, wd = weights(E, I, H, 3), weights(E, I, H, 4), weights(E, H, I, 5)
        tw = torch.softmax(normal((n, K), 6, 1.0, torch.float32), 1).contiguous()
        zero = torch.zeros_like(x)
        new = lambda *shape: torch.empty(shape, device="cuda")
        xs, xn, comb, out, nxt = (torch.empty_like(x) for _ in range(5))
        ep.ep_residual_norm(g, zero, x, xs, xn, wn)
        ep.ep_dispatch(h, xn)
        view = ep.ep_handle_get_buffer(h, A.EP_BUF_HT_STAGE2 if mode == "ht" else A.EP_BUF_LL_RECV)
        rows = view[:r.rows] if mode == "ht" else view
        a, y = out_tensor(r, I), out_tensor(r, H)
        ep.ep_expert_gated(h, rows, wg, wu, a)
        ep.ep_expert_linear(h, a, wd, y)
        ep.ep_combine(h, y, tw, comb)
        ep.ep_residual_norm(g, comb, xs, out, nxt, wn)

        work = torch.empty(ep.ep_residual_norm_workspace(g, n), dtype=torch.uint8, device="cuda")
        gs, gc, dxn, dx, dz = (torch.empty_like(x) for _ in range(5))
        dwn, unused, dtw = new(H), new(H), torch.empty_like(tw)
        ep.ep_residual_norm_backward(g, comb, out, up, zero, wn, gs, gc, unused, work)
        dy, da, dg, du, dr = out_tensor(r, H), out_tensor(r, I), out_tensor(r, I), out_tensor(r, I), out_tensor(r, H)
        ep.ep_combine_backward(h, gc, tw, dy, expert_out=y, grad_weights=dtw)
        dwg, dwu, dwd = new(E, I, H), new(E, I, H), new(E, H, I)
        ep.ep_expert_linear_backward(h, a, wd, dy, grad_x=da, grad_w=dwd)
        ep.ep_expert_gated_backward(h, rows, wg, wu, da, dg, du, grad_rows=dr, grad_w_gate=dwg, grad_w_up=dwu)
        ep.ep_dispatch_backward(h, dr, dxn)
        ep.ep_residual_norm_backward(g, zero, xs, gs, dxn, wn, dx, dz, dwn, work)
        torch.cuda.synchronize()
        assert ep.ep_get_device_error(g) == 0

        point = [t.to("cpu", D) for t in (x, wn, wg, wu, wd, tw)]
        leaves = [t.clone().requires_grad_() for t in point]
        U = up.to("cpu", D)

        def value(p):
            return (block_reference(r, *p[:5], r.topk, p[5]) * U).sum()
        value(leaves).backward()
        for k, (got, what) in enumerate(((dx, "x"), (dwn, "norm weights"), (dwg, "gate weights"), (dwu, "up weights"),
                                         (dwd, "down weights"), (dtw, "routing weights"))):
            check(got.cpu(), leaves[k].grad, lambda t: value([*point[:k], t, *point[k + 1:]]), point[k], 10 * HALF, what)
