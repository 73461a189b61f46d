"""Backward passes of the experts' products from rows kept in 8 bits (ep_expert_gated_backward_fp8 and
ep_expert_linear_backward_fp8).

Their operands are bf16_rne(code * scale), which lie in the rows' gradient meanwhile: the results have the bits of the BF16 calls on those values, whatever the
sizes, and against the 64-bit formula at code * scale an operand's rounding, 2^-8 of it, comes on top of the bounds in
expert_util.
"""
import numpy as np
import pytest
import torch

from expert_util import BF16, D, FP8, HALF, Routing, act64, near, normal, out_tensor, product, row_tensor, untouched
from gpu_util import A, ep, need_gpu, say
from gradient_util import check
from order_util import Ranks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# (mode, sources, tokens per source, experts, top-k, hidden, inner, experts left out): every tile, in HT and in LL with
# one source, few and many; row tiles of every fill; one row; empty experts
SHAPES = [
    ("ht", 1, 1, 8, 1, 128, 8, ()),
    ("ht", 3, 37, 16, 2, 384, 136, (0, 5)),
    ("ll", 4, 33, 16, 3, 512, 264, (15,)),
    ("ll", 16, 9, 32, 3, 256, 136, (31,)),
    ("ll", 1, 50, 8, 2, 1152, 520, ()),
    ("ht", 1, 300, 3, 1, 640, 1000, (0, 2)),
    ("ht", 1, 700, 4, 2, 256, 712, ()),
    ("ht", 1, 2400, 32, 2, 2048, 2072, (7,)),
    ("ll", 4, 600, 32, 2, 2048, 2072, (7,)),
    ("ll", 24, 100, 48, 2, 2048, 1040, (7,)),
    ("ht", 1, 5000, 16, 3, 1920, 1288, (3,)),
]


def weights(E, N, K, seed, pad=0):
    w = torch.full((E, N, K + pad), float("nan"), dtype=BF16, device="cuda")[:, :, :K]
    w.copy_(normal((E, N, K), seed, K ** -0.5))
    return w


def coded(r, C, seed, pad=0, packed=False):
    """Codes and scales of normal rows, NaN in the rows that hold nothing; with `packed` one U8 tensor of both.  Returns
    also the values in 64 bits and rounded to bf16."""
    x = normal((r.rows, C), seed, 2.0, torch.float32)
    s = x.view(r.rows, -1, 128).abs().amax(2) / 448
    q = (x / s.repeat_interleave(128, 1)).to(FP8).view(torch.uint8)
    values = q.view(FP8).to(D) * s.to(D).repeat_interleave(128, 1)
    rounded = (q.view(FP8).float() * s.repeat_interleave(128, 1)).to(BF16)
    rounded[r.unused] = float("nan")
    q[r.unused], s[r.unused] = 0x7F, float("nan")
    if packed:
        used = C + C // 32
        t = torch.full((r.rows, -(-used // 128) * 128 + 16 * pad), 0x7F, dtype=torch.uint8, device="cuda")[:, :used]
        t[:, :C], t[:, C:] = q, s.contiguous().view(torch.uint8)
        return t, None, values, rounded
    wide = torch.full((r.rows, C + 16 * pad), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :C] = q
    more = torch.full((r.rows, C // 128 + pad), float("nan"), device="cuda")
    more[:, :C // 128] = s
    return wide.view(FP8)[:, :C], more[:, :C // 128], values, rounded


def same(a, b, what):
    assert torch.equal(a.view(torch.int16 if a.dtype == BF16 else torch.int32),
                       b.view(torch.int16 if b.dtype == BF16 else torch.int32)), what


def gated_backward(r, I, x, s, wg, wu, dh, gtype, act, coded_rows=True):
    dg, du, dx = out_tensor(r, I, pad=8), out_tensor(r, I), out_tensor(r, r.H)
    g1, g2 = (torch.full((r.E, I, r.H), 9.0, dtype=gtype, device="cuda") for _ in range(2))
    if coded_rows:
        ep.ep_expert_gated_backward_fp8(r.handle, x, wg, wu, dh, dg, du, activation=act, rows_scales=s, grad_rows=dx,
                                        grad_w_gate=g1, grad_w_up=g2)
    else:
        ep.ep_expert_gated_backward(r.handle, x, wg, wu, dh, dg, du, activation=act, grad_rows=dx, grad_w_gate=g1,
                                    grad_w_up=g2)
    return dg, du, dx, g1, g2


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("form,act,gtype", [("packed", "silu", BF16), ("codes", "gelu_tanh", torch.float32)],
                         ids=["packed", "codes"])
def test_gated_backward_has_the_bits_of_the_rounded_rows(shape, form, act, gtype):
    mode, S, T, E, K, H, I, skip = shape
    say(f"gated backward from 8 bits {shape} {form} {act}")
    payload = "fp8" if form == "packed" else "bf16"
    with Routing(mode, S, T, E, K, H, payload=payload, seed=8, skip=skip) as r:
        x, s, _, rounded = coded(r, H, 2, pad=1, packed=form == "packed")
        dh, wg, wu = row_tensor(r, I, 5), weights(E, I, H, 3), weights(E, I, H, 4, pad=8)
        got = gated_backward(r, I, x, s, wg, wu, dh, gtype, act)
        want = gated_backward(r, I, rounded, None, wg, wu, dh, gtype, act, coded_rows=False)
        for a, b, what in zip(got, want, ("gate", "up", "rows", "gate weights", "up weights")):
            same(a, b, what)
        for t in got[:3]:
            untouched(r, t)
        assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("shape", [s[:6] + (i, s[7]) for s, i in
                                   zip(SHAPES, (128, 256, 384, 256, 128, 640, 512, 2048, 1920, 1024, 1280))], ids=str)
@pytest.mark.parametrize("gtype", [BF16, torch.float32], ids=["bf16", "f32"])
def test_linear_backward_has_the_bits_of_the_rounded_rows(shape, gtype):
    mode, S, T, E, K, H, I, skip = shape
    say(f"linear backward from 8 bits {shape} {gtype}")
    with Routing(mode, S, T, E, K, H, seed=7, skip=skip) as r:
        q, s, _, rounded = coded(r, I, 2, pad=1)
        w, dy = weights(E, H, I, 3, pad=8), row_tensor(r, H, 4)
        dx, dw = out_tensor(r, I), torch.full((E, H, I), 9.0, dtype=gtype, device="cuda")
        ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, grad_x=dx, grad_w=dw)
        dx2, dw2 = out_tensor(r, I), torch.empty_like(dw)
        ep.ep_expert_linear_backward(r.handle, rounded, w, dy, grad_x=dx2, grad_w=dw2)
        same(dx, dx2, "rows")
        same(dw, dw2, "weights")
        untouched(r, dx)


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[2], SHAPES[5], SHAPES[8]], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward_against_64_bits(shape, act):
    mode, S, T, E, K, H, I, skip = shape
    say(f"gated backward from 8 bits against 64, {shape} {act}")
    with Routing(mode, S, T, E, K, H, seed=8, skip=skip) as r:
        q, s, values, _ = coded(r, H, 2)
        dh, wg, wu = row_tensor(r, I, 5), weights(E, I, H, 3), weights(E, I, H, 4)
        dg, du, dx, g1, g2 = gated_backward(r, I, q, s, wg, wu, dh, torch.float32, act)
        for e, at in enumerate(r.expert_rows):
            xe, de = values[at], dh[at].to(D)
            def pre(w):     # an operand's rounding on top of the sum's
                v, b = product(xe, w.to(D))
                return v, b * 1.01 + HALF * (xe.abs() @ w.to(D).abs().t())
            (g, bg), (u, bu) = pre(wg[e]), pre(wu[e])
            f, df = act64(g, act)
            bdf = 1.2 * bg + 2.0 ** -18 * (g.abs() + 1)
            vg, vu = de * u * df, de * f
            near(dg[at], vg, de.abs() * (df.abs() * bu + (u.abs() + bu) * bdf) * (1 + HALF) + HALF * vg.abs() * 1.01 + 1e-30,
                 f"gate of expert {e}")
            near(du[at], vu, de.abs() * (1.2 * bg + 2.0 ** -18 * f.abs()) * (1 + HALF) + HALF * vu.abs() * 1.01 + 1e-30,
                 f"up of expert {e}")
            for got, d in ((g1, dg), (g2, du)):
                v, b = product(d[at].to(D).t(), xe.t())
                near(got[e], v, b * 1.01 + HALF * (d[at].to(D).abs().t() @ xe.abs()) + 1e-30, f"weights of expert {e}")


def test_rows_of_a_dispatch():
    """The rows that an FP8 dispatch left, in LL and HT, and ep_dequantize_rows of them: the same bits."""
    say("rows of a dispatch")
    for mode, S in (("ht", 2), ("ll", 3)):
        with Routing(mode, S, 40, 8, 2, 512, payload="fp8", seed=3) as r:
            ep.ep_dispatch(r.handle, normal((r.n, 512), 1, 3.0))
            rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_HT_STAGE2 if mode == "ht" else A.EP_BUF_LL_RECV)
            rows = rows[:r.rows]
            x = torch.full((r.rows, 512), float("nan"), dtype=BF16, device="cuda")
            dense = rows[~r.unused]
            y = torch.empty((dense.shape[0], 512), dtype=BF16, device="cuda")
            ep.ep_dequantize_rows(r.group, dense, y)
            x[~r.unused] = y
            dh, wg, wu = row_tensor(r, 264, 5), weights(8, 264, 512, 3), weights(8, 264, 512, 4)
            got = gated_backward(r, 264, rows, None, wg, wu, dh, BF16, "silu")
            want = gated_backward(r, 264, x, None, wg, wu, dh, BF16, "silu", coded_rows=False)
            for a, b in zip(got, want):
                same(a, b, mode)


def test_scales_and_codes_of_every_kind():
    """Every code, scales of zero, tiny and huge ones: the operand is code * scale rounded to bf16, subnormal products
    and infinities among them.  One expert, one gradient of 1: dW's columns are the operands themselves."""
    say("every code and scale")
    scales = torch.tensor([0.0, 1.0, 2.0 ** -126, 1e-38, 3e-36, 2.0 ** 100, 7.6e35, 0.37, 448.0 ** -1, 1.0000001])
    n, C = len(scales), 256
    with Routing("ht", 1, n, 1, 1, 16, topk=np.zeros((n, 1), np.int32)) as r:
        codes = torch.arange(256, dtype=torch.uint8).repeat(n, 1)
        codes[(codes & 0x7F) == 0x7F] = 0
        q, s = codes.cuda().view(FP8), scales[:, None].repeat(1, 2).cuda()
        w = torch.zeros((1, 16, C), dtype=BF16, device="cuda")
        for i in range(n):
            dy = torch.zeros((n, 16), dtype=BF16, device="cuda")
            dy[i, 3] = 1
            dw = torch.empty((1, 16, C), device="cuda")
            # the other rows must be finite: 0 * inf is NaN
            si = s.clone()
            si[torch.arange(n) != i] = 0
            ep.ep_expert_linear_backward_fp8(r.handle, q, si, w, dy, torch.empty((n, C), dtype=BF16, device="cuda"), dw)
            want = (q[i].float() * s[i].repeat_interleave(128)).to(BF16).float()
            # the matrix unit may flush bf16 subnormals of its operands
            tiny = want.abs() < 2.0 ** -126
            got = dw[0, 3]
            assert torch.equal(got[~tiny], want[~tiny]), float(s[i, 0])
            assert bool((got[tiny].abs() <= 2.0 ** -126).all())


def test_not_finite_rows():
    """A NaN code or scale stays with its row's gradients and its own columns of its expert's weight gradients."""
    say("NaN in one row")
    E, H, I = 4, 512, 264
    with Routing("ht", 1, 50, E, 2, H, seed=5) as r:
        q, s, _, _ = coded(r, H, 2)
        dh, wg, wu = row_tensor(r, I, 5), weights(E, I, H, 3), weights(E, I, H, 4)
        clean = gated_backward(r, I, q, s, wg, wu, dh, BF16, "silu")
        row = int(r.expert_rows[2][1])
        for spoil in ("code", "scale"):
            q2, s2 = q.view(torch.uint8).clone(), s.clone()
            if spoil == "code":
                q2[row, 130] = 0x7F
                columns = slice(130, 131)
            else:
                s2[row, 1] = float("nan")
                columns = slice(128, 256)
            got = gated_backward(r, I, q2.view(FP8), s2, wg, wu, dh, BF16, "silu")
            others = torch.arange(r.rows, device="cuda") != row
            for a, b in zip(got[:3], clean[:3]):
                same(a[others].contiguous(), b[others].contiguous(), spoil)
                assert not bool(a[row].isfinite().any())
            for a, b in zip(got[3:], clean[3:]):
                keep = [e for e in range(E) if e != 2]
                same(a[keep], b[keep], spoil)
                assert not bool(a[2].isfinite().any())     # the row's gradients of the products are NaN in every column
        # the linear product's gradient is given: only the columns of the code, or of the scale's block
        w, dy = weights(E, 64, H, 6), row_tensor(r, 64, 7)
        base = torch.empty((E, 64, H), device="cuda")
        dx = out_tensor(r, H)
        ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, dx, base)
        dw, dx2 = torch.empty_like(base), out_tensor(r, H)
        ep.ep_expert_linear_backward_fp8(r.handle, q2.view(FP8), s2, w, dy, dx2, dw)
        same(dx, dx2, "rows do not depend on them")
        assert bool(dw[2, :, columns].isnan().all())
        dw[2, :, columns] = base[2, :, columns]
        assert torch.equal(dw, base)


def test_short_tensors_and_no_tokens():
    say("short tensors, no tokens")
    E, H, I = 4, 256, 128
    with Routing("ht", 1, 60, E, 2, H, seed=4) as r:
        keep = 77
        q, s, values, rounded = coded(r, I, 2)
        w, dy = weights(E, H, I, 3), row_tensor(r, H, 5)
        dw, dw2 = torch.empty((E, H, I), device="cuda"), torch.empty((E, H, I), device="cuda")
        for cut in ("codes", "gradient"):
            dx = torch.full((r.rows, I), -7.25, dtype=BF16, device="cuda")
            if cut == "codes":
                ep.ep_expert_linear_backward_fp8(r.handle, q[:keep], s[:keep], w, dy, dx, dw)
            else:
                ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, dx[:keep], dw)
            assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
            dx2 = torch.full((r.rows, I), -7.25, dtype=BF16, device="cuda")
            ep.ep_expert_linear_backward(r.handle, rounded[:keep], w, dy, grad_x=dx2, grad_w=dw2)
            same(dw, dw2, cut)
            same(dx, dx2, cut)
            ep.ep_get_device_error(r.group)
        ep.ep_expert_linear_backward_fp8(r.handle, q[:0], s[:0], w, dy[:0], grad_x=torch.empty((0, I), dtype=BF16, device="cuda"),
                                         grad_w=dw)
        assert not bool(dw.any())
    for mode in ("ht", "ll"):
        with Routing(mode, 2, 0, E, 2, H, seed=1, max_tokens_per_rank=4, topk=np.zeros((0, 2), np.int32)) as r:
            q = torch.zeros((r.rows, H), dtype=torch.uint8, device="cuda").view(FP8)
            s = torch.zeros((r.rows, H // 128), device="cuda")
            w = weights(E, I, H, 1)
            got = gated_backward(r, I, q, s, w, w, out_tensor(r, I), BF16, "silu")
            for t in got[:3]:
                assert bool((t == -7.25).all())
            assert not bool(got[3].any()) and not bool(got[4].any())


def test_far_rows():
    """Codes and scales more than 2^31 bytes behind the first, with any stride; strides of the decoded rows that a tile
    cannot span are refused."""
    say("far rows")
    E, N, C = 8, 128, 256
    with Routing("ht", 1, 300, E, 1, N, seed=2) as r:
        q, s, _, rounded = coded(r, C, 3)
        fq, fs = (1 << 24) + 16, (1 << 22) + 3
        big = torch.empty((300 * fq,), dtype=torch.uint8, device="cuda").as_strided((300, C), (fq, 1))
        big.copy_(q.view(torch.uint8))
        far = torch.empty((300 * fs,), device="cuda").as_strided((300, C // 128), (fs, 1))
        far.copy_(s)
        w, dy = weights(E, N, C, 4), row_tensor(r, N, 5)
        dw, dw2 = torch.empty((E, N, C), device="cuda"), torch.empty((E, N, C), device="cuda")
        fx = 4 * 1024 * 1024 - 8
        dx = torch.empty((300 * fx,), dtype=BF16, device="cuda").as_strided((300, C), (fx, 1))
        dx2 = out_tensor(r, C)
        ep.ep_expert_linear_backward_fp8(r.handle, big.view(FP8), far, w, dy, dx, dw)
        ep.ep_expert_linear_backward(r.handle, rounded, w, dy, grad_x=dx2, grad_w=dw2)
        same(dw, dw2, "far")
        same(dx.contiguous(), dx2, "far")
        too_far = torch.empty((300 << 23,), dtype=BF16, device="cuda").as_strided((300, C), (1 << 23, 1))
        with pytest.raises(ep.EpError) as ei:
            ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, too_far, dw)
        assert ei.value.status == A.EP_ERR_UNSUPPORTED


def refused(status, fn, *args, **kw):
    with pytest.raises(ep.EpError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status, (fn.__name__, ei.value)


def test_refusals():
    say("refusals")
    bad = A.EP_ERR_INVALID_ARGUMENT
    E, H, I = 4, 256, 128
    for payload in ("fp8", "bf16"):
        with Routing("ht", 1, 30, E, 2, H, seed=4, payload=payload) as r:
            x, s, _, rounded = coded(r, H, 2)
            u8, _, _, _ = coded(r, H, 2, packed=True)
            wg, dh = weights(E, I, H, 3), row_tensor(r, I, 5)
            dg, du = out_tensor(r, I), out_tensor(r, I)
            dw = torch.full((E, I, H), 9.0, device="cuda")

            gx = out_tensor(r, H)

            def gated(rows=x, scales=s, w=wg, act="silu", grad_rows=gx, **kw):
                ep.ep_expert_gated_backward_fp8(r.handle, rows, w, w, dh, dg, du, grad_rows, activation=act,
                                                rows_scales=scales, **kw)
            refused(bad, gated, grad_rows=None)
            refused(bad, gated, scales=None)                                # codes without scales
            refused(bad, gated, rows=u8)                                    # packed rows with scales
            refused(bad, gated, rows=rounded)                               # BF16 rows: the other call takes them
            refused(bad, gated, rows=rounded, scales=None)
            if payload == "bf16":
                refused(bad, gated, rows=torch.zeros((r.rows, 2 * H), dtype=torch.uint8, device="cuda"), scales=None)
            refused(bad, gated, rows=u8[:, :H], scales=None)                # narrower than a row
            for t in (s[:-1], s[:, :1], s.double().to(BF16), s.t(), s.view(-1), torch.zeros((r.rows, 4), device="cuda")[:, ::2]):
                refused(bad, gated, scales=t)
            refused(bad, gated, rows=x[:, :128])
            refused(bad, gated, rows=torch.zeros((r.rows, H + 8), dtype=torch.uint8, device="cuda").view(FP8)[:, :H])
            refused(bad, gated, w=wg.to(FP8))
            refused(bad, gated, act=7)
            refused(bad, gated, grad_w_gate=dw)
            refused(bad, gated, grad_rows=out_tensor(r, I))

            q, qs, _, _ = coded(r, I, 2)
            w, dy, dx = weights(E, H, I, 3), row_tensor(r, H, 6), out_tensor(r, I)
            lin = ep.ep_expert_linear_backward_fp8
            refused(bad, lin, r.handle, q, None, w, dy, grad_x=dx)
            refused(bad, lin, r.handle, q, qs, w, dy, grad_x=None)
            refused(bad, lin, r.handle, rounded[:, :I], qs, w, dy, grad_x=dx)
            refused(bad, lin, r.handle, q, qs[:-1], w, dy, grad_x=dx)
            refused(bad, lin, r.handle, q.view(torch.uint8), qs, w, dy, grad_x=dx)
            refused(bad, lin, r.handle, q[:, :64], qs, weights(E, H, 64, 3), dy, grad_x=dx[:, :64])   # half a block
            refused(bad, lin, r.handle, q, qs, w.float(), dy, grad_x=dx)
            refused(bad, lin, r.handle, q, qs, w, dy[:, :128], grad_x=dx)
            torch.cuda.synchronize()
            assert all(bool((t == -7.25).all()) for t in (dg, du, dx, gx)) and bool((dw == 9).all())
            assert ep.ep_get_device_error(r.group) == 0
    g = ep.ep_create_group(mode="ht", num_nodes=2, ranks_per_node=2, num_experts=E, top_k=2, max_nodes_per_token=0,
                           hidden=H, max_tokens_per_rank=4, num_src_ranks=1, payload="bf16", ht_stage2="rank")
    h = ep.ep_create_handle(g, torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
    refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_linear_backward_fp8, h, q, qs, w, dy, grad_x=dx)
    ep.ep_destroy_group(g)
    with Routing("ll", 1, 8, E, 2, H, seed=4) as r:                        # LL tensors hold every slot
        q, qs, _, _ = coded(r, I, 2)
        w, dy = weights(E, H, I, 3), row_tensor(r, H, 6)
        refused(bad, ep.ep_expert_linear_backward_fp8, r.handle, q[:-1], qs, w, dy, grad_x=out_tensor(r, I))


def test_three_dimensions():
    """LL rows, scales and outputs as [E, S*T_max, .]."""
    say("three dimensions")
    E, S, T, C, N = 6, 3, 20, 256, 64
    with Routing("ll", S, T, E, 2, N, seed=6) as r:
        q, s, _, _ = coded(r, C, 2)
        w, dy = weights(E, N, C, 3), row_tensor(r, N, 4)
        dx, dw = out_tensor(r, C), torch.empty((E, N, C), dtype=BF16, device="cuda")
        ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, grad_x=dx, grad_w=dw)
        dx3, dw3 = out_tensor(r, C), torch.empty_like(dw)
        shape = lambda t: t.view(E, S * T, t.shape[1])
        ep.ep_expert_linear_backward_fp8(r.handle, shape(q.contiguous()), shape(s.contiguous()), w, shape(dy), grad_x=shape(dx3),
                                         grad_w=dw3)
        same(dx, dx3, "rows")
        same(dw, dw3, "weights")


@pytest.mark.parametrize("mode,S,T,E", [("ht", 1, 90, 6), ("ll", 3, 40, 6), ("ll", 9, 30, 9), ("ht", 1, 1300, 8)])
def test_two_graphs_at_once(mode, S, T, E):
    """Both calls in two graphs of one handle on two streams, replayed on new rows with eager calls between."""
    say(f"two graphs, {mode} {S} x {T}")
    H, I = 384, 256
    with Routing(mode, S, T, E, 2, H, seed=3) as r:
        steps = []
        for k in range(2):
            d = dict(x=coded(r, H, 10 + k)[:2], a=coded(r, I, 20 + k)[:2], dy=row_tensor(r, H, 30 + k), da=out_tensor(r, I),
                     wg=weights(E, I, H, 40 + k), wu=weights(E, I, H, 50 + k), wd=weights(E, H, I, 60 + k),
                     dwd=torch.zeros((E, H, I), device="cuda"), dwg=torch.zeros((E, I, H), dtype=BF16, device="cuda"),
                     dwu=torch.zeros((E, I, H), dtype=BF16, device="cuda"), dg=out_tensor(r, I), du=out_tensor(r, I),
                     dx=out_tensor(r, H))

            def run(d=d):
                ep.ep_expert_linear_backward_fp8(r.handle, *d["a"], d["wd"], d["dy"], grad_x=d["da"], grad_w=d["dwd"])
                ep.ep_expert_gated_backward_fp8(r.handle, d["x"][0], d["wg"], d["wu"], d["da"], d["dg"], d["du"],
                                                rows_scales=d["x"][1], grad_rows=d["dx"], grad_w_gate=d["dwg"],
                                                grad_w_up=d["dwu"])
            steps.append((d, run))
        outs = ("da", "dwd", "dg", "du", "dx", "dwg", "dwu")
        graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
        for d, run in steps:
            run()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run()
            graphs.append(g)
        for turn in range(3):
            want = []
            for k, (d, run) in enumerate(steps):
                for name, C in (("x", H), ("a", I)):
                    q, s = coded(r, C, 100 * turn + k)[:2]
                    d[name][0].view(torch.uint8).copy_(q.view(torch.uint8))
                    d[name][1].copy_(s)
                d["dy"].copy_(row_tensor(r, H, 200 * turn + k))
                run()
                want.append([d[o].clone() for o in outs])
                for o in outs:
                    d[o].fill_(-7.25)
            torch.cuda.synchronize()
            for st, g in zip(streams, graphs):
                with torch.cuda.stream(st):
                    g.replay()
            torch.cuda.synchronize()
            for (d, _), w in zip(steps, want):
                for o, b in zip(outs, w):
                    same(d[o], b, (turn, o))
        assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("mode,S,T", [("ht", 1, 9), ("ht", 1, 150), ("ll", 3, 20)])
def test_gradients_by_differences(mode, S, T, act):
    """Every gradient against differences of the 64-bit formula at the bf16 operands, along directions in which a mistake
    shows (gradient_util).  Bounds: those of the BF16 products' test, the operands being bf16 values as there."""
    say(f"gradients by differences, {mode} {S} x {T}, {act}")
    E, H, I, N = 3, 128, 40, 48
    with Routing(mode, S, T, E, 2, H, seed=13) as r:
        q, s, _, rounded = coded(r, H, 1)
        dh, wg, wu = row_tensor(r, I, 4), weights(E, I, H, 2), weights(E, I, H, 3)
        dg, du, dx, d1, d2 = gated_backward(r, I, q, s, wg, wu, dh, torch.float32, act)
        used = torch.cat(r.expert_rows)
        n = [len(t) for t in r.expert_rows]
        X, DA, WG, WU = rounded[used].to(D), dh[used].to(D), wg.to(D), wu.to(D)

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
            # sums of H = 128 products: 2^-17 of the magnitudes, 2^-12 of |x||w| = O(1) values with room
            mg, mu = xe.abs() @ WG[e].abs().t(), xe.abs() @ WU[e].abs().t()
            eg = 1.05 * HALF * pg.abs() + 2.0 ** -16 * de.abs() * (1.2 * (u.abs() + mu) + 1.2 * mg * u.abs() + u.abs())
            eu = 1.05 * HALF * pu.abs() + 2.0 ** -16 * de.abs() * (1.2 * mg + g.abs())
            for k, (v, b) in enumerate(((pg @ WG[e] + pu @ WU[e], eg @ WG[e].abs() + eu @ WU[e].abs()),
                                        (pg.t() @ xe, eg.t() @ xe.abs()), (pu.t() @ xe, eu.t() @ xe.abs()))):
                ref[k].append(v)
                bound[k].append(b + (1.05 * HALF * v.abs() if k == 0 else 0))
        ref = [torch.cat(ref[0]), torch.stack(ref[1]), torch.stack(ref[2])]
        bound = [torch.cat(bound[0]), torch.stack(bound[1]), torch.stack(bound[2])]
        point = [X, WG, WU]
        for k, (got, what) in enumerate(((dx[used], "rows"), (d1, "gate"), (d2, "up"))):
            check(got, ref[k], lambda t: loss(*point[:k], t, *point[k + 1:]), point[k],
                  float(bound[k].norm() / ref[k].norm()) + 2.0 ** -30, what)
        # the linear product's
        w, dy = weights(E, N, H, 5), row_tensor(r, N, 6)
        dxl, dw = out_tensor(r, H), torch.empty((E, N, H), device="cuda")
        ep.ep_expert_linear_backward_fp8(r.handle, q, s, w, dy, grad_x=dxl, grad_w=dw)
        DY, W = dy[used].to(D), w.to(D)

        def linear(X, W):
            return sum(float(((xe @ W[e].t()) * de).sum()) for e, (xe, de) in enumerate(zip(X.split(n), DY.split(n))))
        parts = list(zip(X.split(n), DY.split(n)))
        rx = torch.cat([de @ W[e] for e, (_, de) in enumerate(parts)])
        bx = torch.cat([N * 2.0 ** -24 * (de.abs() @ W[e].abs()) for e, (_, de) in enumerate(parts)]) + 1.05 * HALF * rx.abs()
        rw = torch.stack([de.t() @ xe for xe, de in parts])
        bw = torch.stack([len(xe) * 2.0 ** -24 * (de.abs().t() @ xe.abs()) for xe, de in parts])
        check(dxl[used], rx, lambda t: linear(t, W), X, float(bx.norm() / rx.norm()) + 2.0 ** -30, "linear rows")
        check(dw, rw, lambda t: linear(X, t), W, float(bw.norm() / rw.norm()) + 2.0 ** -30, "linear weights")


@pytest.mark.parametrize("payload", ["fp8", "bf16"])
@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_training_step_of_the_per_rank_layout(payload, captured):
    """Dispatch, rows into expert order, experts, 8-bit checkpoints, rows back, combine; then the whole chain backward
    from the checkpoints.  Against the 64-bit block that takes the dispatched rows and the checkpoints as they were
    rounded to 8 bits (straight through): 10 bf16 tensors on the longest path, each off by 2^-8 of itself at most with
    errors of random sign, bound the 2-norm of a gradient's difference by 10 2^-8 of it."""
    say(f"training step of the per-rank layout, {payload}, {'captured' if captured else 'eager'}")
    S, T, E, K, H, I = 2, 30, 16, 4, 256, 128
    with Ranks(S=S, T=T, E=E, K=K, H=H, nodes=2, per_node=2, payload=payload, seed=11, max_handles=2) as r:
        n, P = r.n, r.n * K
        x, up = normal((n, H), 1), normal((n, H), 7)
        wg, wu, wd = (normal((E, *sh), 2 + i, sh[1] ** -0.5) for i, sh in enumerate(((I, H), (I, H), (H, I))))
        tw = torch.softmax(normal((n, K), 6, 1.0, torch.float32), 1).contiguous()
        kw = {}
        wgf, wuf = wg, wu
        if payload == "fp8":     # weights that E4M3 holds with a scale of 2^-7: BF16 and FP8 ones are the same values
            step = 2.0 ** -7
            wgf, wuf = (wg / step).to(FP8), (wu / step).to(FP8)
            wg, wu = (wgf.float() * step).to(BF16), (wuf.float() * step).to(BF16)
            one = torch.full((E, 1, H // 128), step, device="cuda")
            kw = dict(w_gate_scales=one, w_up_scales=one)
        new = lambda rows, cols, dtype=BF16: torch.zeros((rows, cols), dtype=dtype, device="cuda")
        u8 = lambda rows, cols: torch.zeros((rows, cols), dtype=torch.uint8, device="cuda").view(FP8)
        pitch = (H + H // 32 + 127) // 128 * 128
        t = dict(sorted=new(P, pitch, torch.uint8) if payload == "fp8" else new(P, H), a=new(P, I), y=new(P, H), qa=u8(P, I),
                 sa=new(P, I // 128, torch.float32), qx=u8(P, H), sx=new(P, H // 128, torch.float32), part=new(P, H),
                 out=new(n, H), gp=new(P, H), gy=new(P, H), gtw=torch.zeros_like(tw), da=new(P, I), dg=new(P, I), du=new(P, I),
                 dxs=new(P, H), dxr=new(P, H), dx=new(n, H), dwd=torch.zeros((E, H, I), device="cuda"),
                 dwg=torch.zeros((E, I, H), device="cuda"), dwu=torch.zeros((E, I, H), device="cuda"))

        def step(h):
            ep.ep_dispatch(h, x)
            rows = ep.ep_handle_get_buffer(h, A.EP_BUF_HT_STAGE2)
            ep.ep_expert_sort(h, rows if payload == "fp8" else rows[:, :2 * H].view(BF16), t["sorted"])
            ep.ep_expert_gated(h, t["sorted"], wgf, wuf, t["a"], **kw)
            if payload == "bf16":
                ep.ep_expert_quantize(h, t["sorted"], t["qx"], t["sx"])
            ep.ep_expert_quantize(h, t["a"], t["qa"], t["sa"])
            ep.ep_expert_linear(h, t["a"], wd, t["y"])
            ep.ep_expert_unsort(h, t["y"], tw, t["part"])
            ep.ep_combine(h, t["part"], None, t["out"])
            ep.ep_combine_backward(h, up, None, t["gp"])
            ep.ep_expert_unsort_backward(h, t["gp"], tw, t["gy"], expert_out=t["y"], grad_weights=t["gtw"])
            ep.ep_expert_linear_backward_fp8(h, t["qa"], t["sa"], wd, t["gy"], grad_x=t["da"], grad_w=t["dwd"])
            saved = dict(rows=t["sorted"]) if payload == "fp8" else dict(rows=t["qx"], rows_scales=t["sx"])
            ep.ep_expert_gated_backward_fp8(h, w_gate=wg, w_up=wu, grad_out=t["da"], grad_gate=t["dg"], grad_up=t["du"],
                                            grad_rows=t["dxs"], grad_w_gate=t["dwg"], grad_w_up=t["dwu"], **saved)
            ep.ep_expert_sort_backward(h, t["dxs"], t["dxr"])
            ep.ep_dispatch_backward(h, t["dxr"], t["dx"])

        if captured:
            step(r.handle)
            eager = {k: v.clone() for k, v in t.items()}
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                h = ep.ep_create_handle(r.group, r.idx)
                step(h)
            for turn in range(3):
                for v in t.values():
                    v.zero_()
                graph.replay()
                torch.cuda.synchronize()
                for k, v in t.items():
                    assert torch.equal(v.view(torch.uint8), eager[k].view(torch.uint8)), (turn, k)
            return
        step(r.handle)
        torch.cuda.synchronize()
        assert ep.ep_get_device_error(r.group) == 0

        deq = lambda q, s: q.to(D) * s.to(D).repeat_interleave(128, 1)
        # the rows as the experts saw them, and as the backward pass saw them
        if payload == "fp8":
            saved = deq(t["sorted"][:, :H].contiguous().view(FP8), t["sorted"][:, H:H + H // 32].contiguous().view(torch.float32))
            seen = saved
        else:
            saved, seen = deq(t["qx"], t["sx"]), t["sorted"].to(D)
        expert, token = r.idx.view(-1).long()[r.entry], r.entry // K
        W1, W2, W3, TW, UP = (v.to(D) for v in (wg, wu, wd, tw, up))
        w = TW.view(-1)[r.entry]

        def experts(X):
            a = torch.empty((P, I), dtype=D, device="cuda")
            parts = [None] * 4
            g, u = torch.empty_like(a), torch.empty_like(a)
            for e in range(E):
                at = expert == e
                g[at], u[at] = X[at] @ W1[e].t(), X[at] @ W2[e].t()
            f, df = act64(g, "silu")
            return g, u, f, df
        g, u, f, df = experts(seen)
        y = torch.stack([(f * u)[i] @ W3[expert[i]].t() for i in range(P)])
        out = torch.zeros((n, H), dtype=D, device="cuda").index_add_(0, token, y * w[:, None])

        def close(got, ref, what):
            rel = float((got.to(D) - ref).norm() / ref.norm())
            assert rel < 10 * HALF, f"{what}: {rel}"
        close(t["out"], out, "output")
        gy = UP[token] * w[:, None]
        gtw = torch.zeros(P, dtype=D, device="cuda")
        gtw[r.entry] = (UP[token] * y).sum(1)
        close(t["gtw"].view(-1), gtw, "routing weights")
        da = torch.stack([gy[i] @ W3[expert[i]] for i in range(P)])
        g, u, f, df = experts(saved)
        dg, du = da * u * df, da * f
        qa = deq(t["qa"], t["sa"])
        dx = torch.stack([dg[i] @ W1[expert[i]] + du[i] @ W2[expert[i]] for i in range(P)])
        close(t["dx"], torch.zeros((n, H), dtype=D, device="cuda").index_add_(0, token, dx), "tokens")
        for name, left, right in (("dwd", gy, qa), ("dwg", dg, saved), ("dwu", du, saved)):
            ref = torch.zeros(t[name].shape, dtype=D, device="cuda")
            for e in range(E):
                at = expert == e
                ref[e] = left[at].t() @ right[at]
            close(t[name], ref, name)
        # the checkpoints are within half a step of what they keep: 2^-4 of a value, or of the smallest code's step
        for q, s, v in ((t["qa"], t["sa"], t["a"]),) + (((t["qx"], t["sx"], t["sorted"]),) if payload == "bf16" else ()):
            near(deq(q, s), v.to(D), 2.0 ** -4 * 1.01 * v.to(D).abs() + 2.0 ** -9 * s.to(D).repeat_interleave(128, 1), "checkpoint")
