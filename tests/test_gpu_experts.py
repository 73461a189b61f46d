"""The experts' products (ep_expert_gated, ep_expert_linear and their backward passes) against 64-bit references.

Rows that hold no message are NaN in every input and must stay as they were in every output.  Bounds: see
expert_util.
"""
import numpy as np
import pytest
import torch

from expert_util import BF16, D, FP8, HALF, Routing, act64, gated, near, normal, out_tensor, product, product_fp8, \
    row_tensor, untouched
from gpu_util import A, ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def weights(E, N, K, seed, pad=0, gap=0):
    """BF16 [E, N, K] of deviation K^-1/2; pad: extra elements per row, gap: extra rows per expert."""
    w = torch.full((E, N + gap, K + pad), float("nan"), dtype=BF16, device="cuda")[:, :N, :K]
    w.copy_(normal((E, N, K), seed, K ** -0.5))
    return w


def weights_fp8(E, N, K, seed):
    w = normal((E, N, K), seed, K ** -0.5, torch.float32)
    nb = (N + 127) // 128
    p = torch.zeros((E, nb * 128, K), device="cuda")
    p[:, :N] = w
    s = p.view(E, nb, 128, K // 128, 128).abs().amax((2, 4)) / 448
    up = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
    return (w / up).to(FP8), s


# (mode, sources, tokens per source, experts, top-k, hidden, inner, experts left out)
SHAPES = [
    ("ht", 1, 1, 8, 1, 16, 8, ()),            # one token, sizes below one piece
    ("ht", 3, 37, 16, 2, 272, 136, (0, 5)),   # contracted tails, empty experts
    ("ll", 4, 33, 16, 3, 512, 264, (15,)),    # slots of several sources
    ("ll", 16, 9, 32, 3, 256, 136, (31,)),    # a list: more sources than are looked up in the counts
    ("ll", 1, 50, 8, 2, 1040, 520, ()),       # one source: slots in place
    ("ht", 1, 700, 4, 2, 256, 712, ()),       # several row tiles per expert
    ("ll", 2, 300, 2, 2, 336, 512, ()),
    ("ht", 1, 300, 3, 1, 640, 1000, (0, 2)),  # all rows on one expert
    ("ht", 1, 2400, 32, 2, 2064, 2072, (7,)),  # the largest tiles, filled by every number of quarters
    ("ll", 4, 600, 32, 2, 2064, 2072, (7,)),
    ("ll", 24, 100, 48, 2, 2064, 1040, (7,)),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated(shape, act):
    mode, S, T, E, K, H, I, skip = shape
    say(f"gated {shape} {act}")
    with Routing(mode, S, T, E, K, H, seed=1, skip=skip) as r:
        x = row_tensor(r, H, 2, pad=8)
        wg, wu = weights(E, I, H, 3, pad=16), weights(E, I, H, 4, gap=2)
        out = out_tensor(r, I, pad=24)
        ep.ep_expert_gated(r.handle, x, wg, wu, out, activation=act)
        for e, at in enumerate(r.expert_rows):
            if len(at):
                xe = x[at].to(D)
                v, b = gated(product(xe, wg[e].to(D)), product(xe, wu[e].to(D)), act)
                near(out[at], v, b, f"expert {e}")
        untouched(r, out)
        assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("shape", [s[:5] + (h, i, s[7]) for s, h, i in
                                   zip(SHAPES, (128, 384, 512, 256, 1152, 256, 640, 896, 384, 384, 256),
                                       (8, 136, 256, 136, 520, 712, 128, 1000, 2072, 2072, 1040))],
                         ids=str)
def test_gated_fp8(shape):
    """Rows as the dispatch packed them, in the group's own buffer."""
    mode, S, T, E, K, H, I, skip = shape
    say(f"gated FP8 {shape}")
    with Routing(mode, S, T, E, K, H, payload="fp8", seed=1, skip=skip) as r:
        ep.ep_dispatch(r.handle, normal((r.n, H), 2))
        rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_HT_STAGE2 if mode == "ht" else A.EP_BUF_LL_RECV)
        (wg, sg), (wu, su) = weights_fp8(E, I, H, 3), weights_fp8(E, I, H, 4)
        out = out_tensor(r, I)
        ep.ep_expert_gated(r.handle, rows, wg, wu, out, w_gate_scales=sg, w_up_scales=su)
        for e, at in enumerate(r.expert_rows):
            if len(at):
                raw = rows[at]
                q = raw[:, :H].contiguous().view(FP8)
                s = raw[:, H:H + H // 32].contiguous().view(torch.float32)
                v, b = gated(product_fp8(q, s, wg[e], sg[e]), product_fp8(q, s, wu[e], su[e]), "silu")
                near(out[at], v, b, f"expert {e}")
        untouched(r, out)


def test_gated_packed_bf16_rows():
    """A BF16 payload's packed rows and the same rows as a BF16 tensor give the same bits."""
    say("gated on packed BF16 rows")
    with Routing("ll", 2, 40, 8, 2, 256, seed=5) as r:
        ep.ep_dispatch(r.handle, normal((r.n, 256), 2))
        rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_LL_RECV)
        wg, wu = weights(8, 136, 256, 3), weights(8, 136, 256, 4)
        a, b = out_tensor(r, 136), out_tensor(r, 136)
        ep.ep_expert_gated(r.handle, rows, wg, wu, a)
        ep.ep_expert_gated(r.handle, rows[:, :512].contiguous().view(BF16), wg, wu, b)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(shape):
    mode, S, T, E, K, H, I, skip = shape
    say(f"linear {shape}")
    with Routing(mode, S, T, E, K, H, seed=6, skip=skip) as r:
        x, w, out = row_tensor(r, I, 2), weights(E, H, I, 3), out_tensor(r, H)
        ep.ep_expert_linear(r.handle, x, w, out)
        for e, at in enumerate(r.expert_rows):
            if len(at):
                v, b = product(x[at].to(D), w[e].to(D))
                near(out[at], v, b + HALF * v.abs() * 1.01, f"expert {e}")
        untouched(r, out)


@pytest.mark.parametrize("shape", [s[:6] + (i, s[7]) for s, i in zip(SHAPES, (128, 256, 384, 256, 128, 640, 512, 1024, 384, 384, 256))],
                         ids=str)
def test_linear_fp8(shape):
    mode, S, T, E, K, H, I, skip = shape
    say(f"linear FP8 {shape}")
    with Routing(mode, S, T, E, K, H, seed=6, skip=skip) as r:
        x = normal((r.rows, I), 2, 3.0, torch.float32)
        xs = x.view(r.rows, -1, 128).abs().amax(2) / 448
        q = (x / xs.repeat_interleave(128, 1)).to(FP8)
        q[r.unused] = torch.full((), float("nan"), device="cuda").to(FP8)
        w, ws = weights_fp8(E, H, I, 3)
        out = out_tensor(r, H)
        ep.ep_expert_linear(r.handle, q, w, out, x_scales=xs, w_scales=ws)
        for e, at in enumerate(r.expert_rows):
            if len(at):
                v, b = product_fp8(q[at], xs[at], w[e], ws[e])
                near(out[at], v, b + HALF * v.abs() * 1.01, f"expert {e}")
        untouched(r, out)


def check_weight_grad(r, got, dy, x, what):
    for e, at in enumerate(r.expert_rows):
        v, b = product(dy[at].to(D).t(), x[at].to(D).t())
        near(got[e], v, b + (HALF * v.abs() * 1.01 if got.dtype == BF16 else 0) + 1e-30, f"{what} of expert {e}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("wtype", [BF16, torch.float32], ids=["bf16", "f32"])
def test_linear_backward(shape, wtype):
    mode, S, T, E, K, H, I, skip = shape
    say(f"linear backward {shape} {wtype}")
    with Routing(mode, S, T, E, K, H, seed=7, skip=skip) as r:
        x, w, dy = row_tensor(r, I, 2), weights(E, H, I, 3, pad=8), row_tensor(r, H, 4)
        dx = out_tensor(r, I)
        dw = torch.full((E, H, I), 9.0, dtype=wtype, device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, w, dy, grad_x=dx, grad_w=dw)
        for e, at in enumerate(r.expert_rows):
            if len(at):
                v, b = product(dy[at].to(D), w[e].to(D).t())
                near(dx[at], v, b + HALF * v.abs() * 1.01, f"rows of expert {e}")
        untouched(r, dx)
        check_weight_grad(r, dw, dy, x, "weights")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward(shape, act):
    mode, S, T, E, K, H, I, skip = shape
    say(f"gated backward {shape} {act}")
    with Routing(mode, S, T, E, K, H, seed=8, skip=skip) as r:
        x, dh = row_tensor(r, H, 2), row_tensor(r, I, 5)
        wg, wu = weights(E, I, H, 3), weights(E, I, H, 4, pad=8)
        dg, du, dx = out_tensor(r, I, pad=8), out_tensor(r, I), out_tensor(r, H)
        dwg = torch.full((E, I, H), 9.0, dtype=BF16, device="cuda")
        dwu = torch.full((E, I, H), 9.0, dtype=BF16, device="cuda")
        ep.ep_expert_gated_backward(r.handle, x, wg, wu, dh, dg, du, activation=act, grad_rows=dx, grad_w_gate=dwg,
                                    grad_w_up=dwu)
        for e, at in enumerate(r.expert_rows):
            if not len(at):
                continue
            xe, de = x[at].to(D), dh[at].to(D)
            (g, bg), (u, bu) = product(xe, wg[e].to(D)), product(xe, wu[e].to(D))
            f, df = act64(g, act)
            # |act''| <= 1.1; the derivative's own terms cancel near its zeros: 2^-18 of |g| + 1
            bdf = 1.2 * bg + 2.0 ** -18 * (g.abs() + 1)
            vg, vu = de * u * df, de * f
            near(dg[at], vg, de.abs() * (df.abs() * bu + (u.abs() + bu) * bdf) + HALF * vg.abs() * 1.01 + 1e-30,
                 f"gate of expert {e}")
            near(du[at], vu, de.abs() * (1.2 * bg + 2.0 ** -18 * f.abs()) + HALF * vu.abs() * 1.01 + 1e-30,
                 f"up of expert {e}")
            # the other products read the bf16 gradients that were given back
            (a, ba), (b, bb) = product(dg[at].to(D), wg[e].to(D).t()), product(du[at].to(D), wu[e].to(D).t())
            near(dx[at], a + b, 2 * (ba + bb) + HALF * (a + b).abs() * 1.01, f"rows of expert {e}")
        for t in (dg, du, dx):
            untouched(r, t)
        check_weight_grad(r, dwg, dg, x, "gate weights")
        check_weight_grad(r, dwu, du, x, "up weights")
