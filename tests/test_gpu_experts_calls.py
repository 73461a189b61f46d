"""Calls of the experts' products other than the plain one: refusals, tensors that are too short, strides, far
offsets, repeated entries, other streams, captured graphs, and the whole block as a training step and as a
decode step run it.  Bounds: see expert_util.
"""
import pytest
import torch

from expert_util import BF16, D, FP8, HALF, Routing, act64, gated, near, normal, out_tensor, product, row_tensor, untouched
from gpu_util import A, ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def weights(E, N, K, seed):
    return normal((E, N, K), seed, K ** -0.5)


def check_linear(r, x, w, out, experts=None):
    for e, at in enumerate(r.expert_rows):
        if len(at) and (experts is None or e in experts):
            v, b = product(x[at].to(D), w[e].to(D))
            near(out[at], v, b + HALF * v.abs() * 1.01, f"expert {e}")


def refused(status, call, *a, **kw):
    with pytest.raises(ep.EpError) as e:
        call(*a, **kw)
    assert e.value.status == status, str(e.value)


def test_refusals():
    """Every call here returns before it enqueues anything: outputs keep their values."""
    say("refusals of the experts' products")
    E, H, I = 8, 256, 136
    bad = A.EP_ERR_INVALID_ARGUMENT
    with Routing("ll", 2, 20, E, 2, H, seed=1) as r, Routing("ht", 1, 20, E, 2, H, payload="fp8", seed=1) as f:
        x, out, dx = row_tensor(r, H, 2), out_tensor(r, I), out_tensor(r, H)
        w = weights(E, I, H, 3)
        wd = weights(E, H, I, 4)
        g = row_tensor(r, I, 5)
        w8, s8 = torch.zeros((E, I, H), dtype=FP8, device="cuda"), torch.zeros((E, 2, 2), device="cuda")
        gw = torch.full((E, I, H), 3.0, dtype=BF16, device="cuda")
        ok = dict(handle=r.handle, rows=x, w_gate=w, w_up=w, out=out)

        def no(status=bad, **kw):
            refused(status, ep.ep_expert_gated, **{**ok, **kw})
        no(rows=x[:-1])                                  # LL tensors hold every slot
        no(out=out[:-1])
        no(rows=x[:, :-16])
        no(rows=x.float())
        no(rows=x.view(E, 2, 20, H)[:, 0])               # an LL view that leaves sources out
        no(w_gate=w[:, :, :-16])
        no(w_gate=w[:-1])
        no(w_gate=w[:, :-8])                             # another size than w_up's
        no(w_gate=w[:, :-4], w_up=w[:, :-4])             # not a multiple of 8
        no(w_gate=w.transpose(1, 2).contiguous().transpose(1, 2))
        no(w_gate=torch.zeros((E, I, H + 4), dtype=BF16, device="cuda")[:, :, :H])   # rows not on 16 bytes
        no(w_gate=w.half())
        no(w_gate_scales=s8, w_up_scales=s8)             # scales with BF16 weights
        no(w_gate=w8, w_up=w8, w_gate_scales=s8, w_up_scales=s8)   # FP8 weights with BF16 rows
        no(activation=2)
        no(out=out.float())
        with pytest.raises(ValueError):
            ep.ep_expert_gated(**{**ok, "activation": "relu"})
        with pytest.raises(ValueError):
            ep.ep_expert_gated(**{**ok, "rows": x.cpu()})
        packed = torch.zeros((f.rows, H + H // 32), dtype=torch.uint8, device="cuda")
        wide = torch.zeros((f.rows, 272), dtype=torch.uint8, device="cuda")
        o8 = torch.full((f.rows, I), -7.25, dtype=BF16, device="cuda")
        ok8 = dict(handle=f.handle, rows=wide[:, :264], w_gate=w8, w_up=w8, out=o8, w_gate_scales=s8, w_up_scales=s8)

        def no8(**kw):
            refused(bad, ep.ep_expert_gated, **{**ok8, **kw})
        no8(rows=packed)                                 # rows of 264 bytes: not on 16
        no8(rows=wide[:, :256])                          # shorter than a packed row
        no8(w_gate_scales=None)
        no8(w_gate_scales=s8[:, :1])
        no8(w_gate_scales=s8[:, :, :1])
        no8(w_gate_scales=s8.to(BF16))
        no8(w_gate=w)
        refused(bad, ep.ep_expert_gated_backward, f.handle, wide[:, :264], w, w, o8, o8, o8)   # FP8 rows

        back = dict(handle=r.handle, rows=x, w_gate=w, w_up=w, grad_out=g, grad_gate=out, grad_up=out_tensor(r, I),
                    grad_rows=dx, grad_w_gate=gw, grad_w_up=gw.clone())

        def nob(**kw):
            refused(bad, ep.ep_expert_gated_backward, **{**back, **kw})
        nob(grad_w_up=None)
        nob(grad_w_up=gw.float())
        nob(grad_w_gate=gw.half(), grad_w_up=gw.half())
        nob(grad_w_gate=gw[:1].expand(E, I, H))          # experts' gradients in one memory
        nob(grad_rows=dx[:, :-8])
        nob(grad_gate=out[:, :-8])
        nob(grad_out=g[:-1])
        lin = dict(handle=r.handle, x=g, w=wd, out=dx)

        def nol(**kw):
            refused(bad, ep.ep_expert_linear, **{**lin, **kw})
        nol(x=x)
        nol(x_scales=s8)
        nol(w=wd.to(FP8))
        nol(x=torch.zeros((r.rows, I), dtype=FP8, device="cuda"), w=wd.to(FP8))   # no scales; 136 is no multiple of 128
        refused(bad, ep.ep_expert_linear_backward, r.handle, g, wd, out)
        torch.cuda.synchronize()
        for t in (out, dx, o8):
            assert bool((t == -7.25).all())
        assert bool((gw == 3.0).all())
    rank = ep.ep_create_group(mode="ht", num_nodes=2, ranks_per_node=2, num_experts=8, top_k=2, max_nodes_per_token=0,
                              hidden=H, max_tokens_per_rank=4, num_src_ranks=1, payload="bf16", ht_stage2="rank")
    h = ep.ep_create_handle(rank, torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda"))
    t = torch.zeros((8, H), dtype=BF16, device="cuda")
    refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_linear, h, t, weights(8, H, H, 1), t.clone())
    ep.ep_destroy_handle(h)
    refused(bad, ep.ep_expert_linear, h, t, weights(8, H, H, 1), t.clone())
    ep.ep_destroy_group(rank)


def test_pending_dispatch_is_refused():
    say("products while a staged dispatch is pending")
    with Routing("ll", 1, 16, 4, 2, 256, seed=3) as r:
        ep.ep_dispatch(r.handle, normal((16, 256), 1), send_only=True)
        rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_LL_RECV)
        w, out = weights(4, 64, 256, 2), out_tensor(r, 64)
        refused(A.EP_ERR_INVALID_ARGUMENT, ep.ep_expert_gated, r.handle, rows, w, w, out)
        ep.ep_complete(r.handle)
        ep.ep_expert_gated(r.handle, rows, w, w, out)
        untouched(r, out)


def test_rows_beyond_the_tensors():
    """HT rows that the tensors do not hold are left out of every product and reported."""
    say("tensors shorter than the received rows")
    E, H, I = 4, 256, 72
    with Routing("ht", 1, 60, E, 2, H, seed=4) as r:
        keep = 77                                            # of 120 rows: ends inside an expert
        x, w = row_tensor(r, I, 2), weights(E, H, I, 3)
        big = torch.full((r.rows, H), -7.25, dtype=BF16, device="cuda")
        ep.ep_expert_linear(r.handle, x, w, big[:keep])
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        assert bool((big[keep:] == -7.25).all())
        whole = torch.empty_like(big)
        ep.ep_expert_linear(r.handle, x, w, whole)
        assert ep.ep_get_device_error(r.group) == 0
        assert torch.equal(whole[:keep], big[:keep])
        dy = row_tensor(r, H, 5)
        dw = torch.empty((E, H, I), device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, w, dy[:keep], grad_w=dw)
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        for e, at in enumerate(r.expert_rows):
            at = at[at < keep]
            v, b = product(dy[at].to(D).t(), x[at].to(D).t())
            near(dw[e], v, b + 1e-30, f"expert {e}")
        none = torch.empty((0, H), dtype=BF16, device="cuda")
        ep.ep_expert_linear(r.handle, x, w, none)
        ep.ep_expert_linear_backward(r.handle, x, w, none, grad_w=dw)
        assert bool((dw == 0).all())
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE


@pytest.mark.parametrize("mode", ["ht", "ll"])
def test_no_tokens(mode):
    """A batch of no tokens: nothing is written, gradients of weights are zeros."""
    say(f"products of an empty batch, {mode}")
    E, H, I = 8, 256, 64
    with Routing(mode, 2, 0, E, 2, H, seed=1, max_tokens_per_rank=4,
                 topk=torch.zeros((0, 2), dtype=torch.int32).numpy()) as r:
        x, out = out_tensor(r, H), out_tensor(r, I)
        w = weights(E, I, H, 1)
        dw = torch.full((E, I, H), 9.0, dtype=BF16, device="cuda")
        ep.ep_expert_gated(r.handle, x, w, w, out)
        ep.ep_expert_gated_backward(r.handle, x, w, w, out, out_tensor(r, I), out_tensor(r, I), grad_rows=x,
                                    grad_w_gate=dw, grad_w_up=dw.clone())
        assert bool((out == -7.25).all()) and bool((x == -7.25).all()) and bool((dw == 0).all())


def test_invalid_entries():
    """Entries outside the experts and repeated ones have no row and take part in nothing."""
    say("products after a routing with invalid entries")
    import numpy as np
    rng = np.random.default_rng(3)
    topk = np.argsort(rng.random((90, 16)), axis=1)[:, :4].astype(np.int32)
    topk[5, 1], topk[8, 3], topk[20] = -1, 16, 99
    topk[30, 2] = topk[30, 0]
    for mode, S in (("ht", 1), ("ll", 3)):
        with Routing(mode, S, 90 // S, 16, 4, 256, topk=topk) as r:
            x, w, out = row_tensor(r, 128, 1), weights(16, 256, 128, 2), out_tensor(r, 256)
            ep.ep_expert_linear(r.handle, x, w, out)
            check_linear(r, x, w, out)
            untouched(r, out)


def test_far_offsets():
    """Rows and weights further apart than 2^31 bytes and elements, one expert's weights for all (stride 0)."""
    say("far offsets")
    E, N, K = 8, 128, 64
    with Routing("ht", 1, 300, E, 1, N, seed=2) as r:
        far = 4 * 1024 * 1024 - 8                            # elements between rows: 300 rows span 2.5 GB
        x = torch.empty((300 * far + K,), dtype=BF16, device="cuda").as_strided((300, K), (far, 1))
        x.copy_(normal((300, K), 3))
        w = torch.empty((E * (1 << 28),), dtype=BF16, device="cuda").as_strided((E, N, K), (1 << 28, 1024, 1))
        w.copy_(weights(E, N, K, 4))
        out = torch.empty((300 * far + N,), dtype=BF16, device="cuda").as_strided((300, N), (far, 1))
        ep.ep_expert_linear(r.handle, x, w, out)
        check_linear(r, x, w, out)
        one = w[3:4].expand(E, N, K)
        ep.ep_expert_linear(r.handle, x, one, out)
        check_linear(r, x, one, out)
        dx = torch.empty((300, K), dtype=BF16, device="cuda")
        dw = torch.empty((E, N, K), device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, w, out, grad_x=dx, grad_w=dw)
        for e, at in enumerate(r.expert_rows):
            v, b = product(out[at].to(D), w[e].to(D).t())
            near(dx[at], v, b + HALF * v.abs() * 1.01, f"rows of {e}")
            v, b = product(out[at].to(D).t(), x[at].to(D).t())
            near(dw[e], v, b + 1e-30, f"weights of {e}")
        too_far = torch.empty((300 << 23,), dtype=BF16, device="cuda").as_strided((300, K), (1 << 23, 1))
        refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_linear, r.handle, too_far, w, out)


def test_not_finite_values_stay_in_their_rows():
    say("infinity and NaN in one row")
    E, H, I = 4, 512, 264
    with Routing("ht", 1, 50, E, 2, H, seed=5) as r:
        x, w, clean = row_tensor(r, H, 2), weights(E, I, H, 3), out_tensor(r, I)
        ep.ep_expert_gated(r.handle, x, w, w, clean)
        x[7, 3], x[40, 511] = float("inf"), float("nan")
        out = out_tensor(r, I)
        ep.ep_expert_gated(r.handle, x, w, w, out)
        same = torch.ones(r.rows, dtype=torch.bool, device="cuda")
        same[[7, 40]] = False
        assert torch.equal(out[same], clean[same])
        assert not bool(out[40].isfinite().any()) and not bool(out[7].isfinite().all())


@pytest.mark.parametrize("tokens", [30, 400])
def test_repeated_and_on_another_stream(tokens):
    """The same bits again, on the caller's stream behind its other work, with two handles of one group in turn."""
    say(f"repeated calls on a stream of their own, {tokens} tokens")
    E, H, I = 8, 512, 384
    with Routing("ll", 4, tokens // 2, E, 2, H, seed=6) as r:
        x, dy, w = row_tensor(r, H, 2), row_tensor(r, I, 3), weights(E, I, H, 4)
        topk2 = r.idx.flip(0).contiguous()
        h2 = ep.ep_create_handle(r.group, topk2)
        first = None
        for turn in range(3):
            s = torch.cuda.Stream()
            late = torch.zeros_like(x)
            out, dx = out_tensor(r, I), out_tensor(r, H)
            dw = torch.empty((E, I, H), device="cuda")
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
                late.copy_(x)
                ep.ep_expert_linear(h2, late, w, out_tensor(r, I))
                ep.ep_expert_linear(r.handle, late, w, out)
                ep.ep_expert_linear_backward(r.handle, late, w, dy, grad_x=dx, grad_w=dw)
            s.synchronize()
            got = [t.clone() for t in (out, dx, dw)]
            first = first or got
            assert all(torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0)) for a, b in zip(first, got)), turn
        check_linear(r, x, w, first[0])
        ep.ep_destroy_handle(h2)


@pytest.mark.parametrize("mode,S", [("ht", 2), ("ll", 1), ("ll", 3)])
def test_quantize_rows(mode, S):
    """Codes and scales are ep_quantize's bit for bit; rows that hold nothing stay; short tensors are reported."""
    say(f"quantised rows, {mode} {S}")
    E, C = 6, 640
    with Routing(mode, S, 40, E, 2, 256, seed=9) as r, Routing("ht", 1, 1, 1, 1, C, payload="fp8") as f:
        x = row_tensor(r, C, 2, 3.0, pad=8)
        x[~r.unused] *= torch.logspace(-30, 20, int((~r.unused).sum()), device="cuda")[:, None]
        x[r.expert_rows[1][0], 128:256] = 0
        used = x[~r.unused].contiguous()
        q0 = torch.empty(used.shape, dtype=FP8, device="cuda")
        s0 = torch.empty((used.shape[0], C // 128), device="cuda")
        ep.ep_quantize(f.group, used, q0, s0)
        q = torch.full((r.rows, C + 16), 7, dtype=torch.uint8, device="cuda").view(FP8)[:, :C]
        s = torch.full((r.rows, C // 128 + 1), -7.25, device="cuda")[:, :C // 128]
        ep.ep_expert_quantize(r.handle, x, q, s)
        assert torch.equal(q[~r.unused].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[~r.unused], s0)
        assert bool((q[r.unused].view(torch.uint8) == 7).all()) and bool((s[r.unused] == -7.25).all())
        assert ep.ep_get_device_error(r.group) == 0
        bad = A.EP_ERR_INVALID_ARGUMENT
        refused(bad, ep.ep_expert_quantize, r.handle, x[:, :C - 64], q[:, :C - 64], s)
        refused(bad, ep.ep_expert_quantize, r.handle, x, q[:, :C - 128], s)
        refused(bad, ep.ep_expert_quantize, r.handle, x, q, s[:, :-1])
        refused(bad, ep.ep_expert_quantize, r.handle, x.float(), q, s)
        refused(bad, ep.ep_expert_quantize, r.handle, x, q.view(torch.uint8), s)
        if mode == "ht":
            ep.ep_expert_quantize(r.handle, x, q[:-1], s)
            assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        else:
            refused(bad, ep.ep_expert_quantize, r.handle, x, q[:-1], s)


def block_reference(r, x, wn, wg, wu, wd, topk, tw, eps=1e-6):
    """The block in 64 bits with gradients: norm, experts, weighted sum, residual, norm."""
    out = []
    xn = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * wn
    for i in range(x.shape[0]):
        acc = 0
        for k in range(topk.shape[1]):
            e = int(topk[i, k])
            g, u = wg[e] @ xn[i], wu[e] @ xn[i]
            acc = acc + tw[i, k] * (wd[e] @ (g * torch.sigmoid(g) * u))
        out.append(acc)
    return x + torch.stack(out)


@pytest.mark.parametrize("mode", ["ht", "ll"])
def test_training_step(mode):
    """Norm, dispatch, experts, combine, residual and norm forward, then the whole chain backward, against 64 bits.

    Every tensor between two calls is bf16: an error of 2^-8 of it at most, of random sign, passes through sums of
    many such terms.  The 2-norm of the difference is bounded by the number of bf16 tensors on the longest path (10)
    times 2^-8 of the result's."""
    say(f"training step, {mode}")
    E, K, H, I, S, T = 8, 2, 256, 128, 2, 12
    n = S * T
    with Routing(mode, S, T, E, K, H, seed=11) as r:
        x = normal((n, H), 1)
        wn = 1 + normal((H,), 2, 0.1, torch.float32)
        wg, wu, wd = weights(E, I, H, 3), weights(E, I, H, 4), weights(E, H, I, 5)
        tw = torch.softmax(normal((n, K), 6, 1.0, torch.float32), 1).contiguous()
        up = normal((n, H), 7)
        h, g = r.handle, r.group
        zero = torch.zeros_like(x)
        xs, xn = torch.empty_like(x), torch.empty_like(x)
        ep.ep_residual_norm(g, zero, x, xs, xn, wn)                       # the norm in front: nothing to add
        ep.ep_dispatch(h, xn)
        view = ep.ep_handle_get_buffer(h, A.EP_BUF_HT_STAGE2 if mode == "ht" else A.EP_BUF_LL_RECV)
        rows = view[:r.rows] if mode == "ht" else view
        a, y = out_tensor(r, I), out_tensor(r, H)
        ep.ep_expert_gated(h, rows, wg, wu, a)
        ep.ep_expert_linear(h, a, wd, y)
        comb = torch.empty_like(x)
        ep.ep_combine(h, y, tw, comb)
        out, nxt = torch.empty_like(x), torch.empty_like(x)
        ep.ep_residual_norm(g, comb, xs, out, nxt, wn)

        # backward from a gradient of the stream and none of the second norm
        gs, gc = torch.empty_like(x), torch.empty_like(x)
        gw2, work = torch.empty(H, device="cuda"), torch.empty(ep.ep_residual_norm_workspace(g, n), dtype=torch.uint8,
                                                               device="cuda")
        ep.ep_residual_norm_backward(g, comb, out, up, zero, wn, gs, gc, gw2, work)
        dy, dtw = out_tensor(r, H), torch.empty_like(tw)
        ep.ep_combine_backward(h, gc, tw, dy, expert_out=y, grad_weights=dtw)
        da, dwd = out_tensor(r, I), torch.empty((E, H, I), device="cuda")
        ep.ep_expert_linear_backward(h, a, wd, dy, grad_x=da, grad_w=dwd)
        dg, du, dr = out_tensor(r, I), out_tensor(r, I), out_tensor(r, H)
        dwg, dwu = torch.empty((E, I, H), device="cuda"), torch.empty((E, I, H), device="cuda")
        ep.ep_expert_gated_backward(h, rows, wg, wu, da, dg, du, grad_rows=dr, grad_w_gate=dwg, grad_w_up=dwu)
        dxn = torch.empty_like(x)
        ep.ep_dispatch_backward(h, dr, dxn)
        dx, dz, dwn = torch.empty_like(x), torch.empty_like(x), torch.empty(H, device="cuda")
        ep.ep_residual_norm_backward(g, zero, xs, gs, dxn, wn, dx, dz, dwn, work)
        torch.cuda.synchronize()
        assert ep.ep_get_device_error(g) == 0

        L = [t.to(D).requires_grad_() for t in (x, wn, wg, wu, wd, tw)]
        want = block_reference(r, *L[:5], r.topk, L[5])
        want.backward(up.to(D))

        def close(got, ref, what):
            rel = float((got.to(D) - ref).norm() / ref.norm())
            assert rel < 10 * HALF, f"{what}: {rel}"
        close(out, want.detach(), "stream")
        for got, leaf, what in ((dx, L[0], "x"), (dwn, L[1], "norm weights"), (dwg, L[2], "gate weights"),
                                (dwu, L[3], "up weights"), (dwd, L[4], "down weights"), (dtw, L[5], "routing weights")):
            close(got, leaf.grad, what)
        # the same against differences of the 64-bit block along a random direction
        with torch.no_grad():
            v = [normal(t.shape, 20 + i, float(t.detach().std()), torch.float32).to(D) for i, t in enumerate(L)]
            step = 1e-5
            f = [float((block_reference(r, *[t + c * step * d for t, d in zip(L[:5], v[:5])], r.topk,
                                        L[5] + c * step * v[5]) * up.to(D)).sum()) for c in (1, -1)]
            diff = (f[0] - f[1]) / (2 * step)
            got = sum(float((t.to(D) * d).sum()) for t, d in zip((dx, dwn, dwg, dwu, dwd, dtw), v))
            size = sum(float(t.to(D).norm() * d.norm()) for t, d in zip((dx, dwn, dwg, dwu, dwd, dtw), v))
            assert abs(got - diff) < 10 * HALF * size, (got, diff, size)


def test_gradients_by_differences():
    """ep_expert_gated_backward and ep_expert_linear_backward against differences of the 64-bit formula."""
    say("gradients by differences")
    E, H, I = 3, 64, 40
    with Routing("ht", 1, 9, E, 2, H, seed=13) as r:
        x, w1, w2, dh = row_tensor(r, H, 1), weights(E, I, H, 2), weights(E, I, H, 3), row_tensor(r, I, 4)
        dg, du, dx = out_tensor(r, I), out_tensor(r, I), out_tensor(r, H)
        d1, d2 = torch.empty((E, I, H), device="cuda"), torch.empty((E, I, H), device="cuda")
        ep.ep_expert_gated_backward(r.handle, x, w1, w2, dh, dg, du, activation="gelu_tanh", grad_rows=dx,
                                    grad_w_gate=d1, grad_w_up=d2)

        def loss(x, w1, w2):
            total = 0.0
            for e, at in enumerate(r.expert_rows):
                f, _ = act64(x[at] @ w1[e].t(), "gelu_tanh")
                total += float((f * (x[at] @ w2[e].t()) * dh[at].to(D)).sum())
            return total
        base = [t.to(D) for t in (x, w1, w2)]
        for k, got in enumerate((dx, d1, d2)):
            for seed in range(3):
                v = normal(got.shape, 30 + seed, 1.0, torch.float32).to(D)
                at = [[t + c * 1e-5 * v if i == k else t for i, t in enumerate(base)] for c in (1, -1)]
                diff = (loss(*at[0]) - loss(*at[1])) / 2e-5
                # dg and du are rounded to bf16 before the products, and dx once more
                size = float(got.to(D).norm() * v.norm())
                assert abs(float((got.to(D) * v).sum()) - diff) < 2 * HALF * size, (k, seed)


@pytest.mark.parametrize("form", ["bf16", "fp8"])
def test_decode_step_in_a_graph(form):
    """Handle, dispatch, experts and combine of an LL decode step captured once and replayed on new inputs, with
    the same calls run eagerly between the replays: every replay equals them bit for bit."""
    say(f"captured decode step, {form}")
    E, K, H, I, S, T = 8, 2, 512, 256, 4, 8
    n = S * T
    kw = dict(mode="ll", num_nodes=2, ranks_per_node=2, num_experts=E, top_k=K, max_nodes_per_token=0, hidden=H,
              max_tokens_per_rank=T, num_src_ranks=S, payload=form)
    one, two = ep.ep_create_group(**kw), ep.ep_create_group(**kw)
    wg, wu, wd = weights(E, I, H, 1), weights(E, I, H, 2), weights(E, H, I, 3)
    sc = {}
    if form == "fp8":
        sc = dict(w_gate_scales=torch.full((E, 2, H // 128), 0.01, device="cuda"),
                  w_up_scales=torch.full((E, 2, H // 128), 0.02, device="cuda"))
        wg, wu = (wg / 0.01).clamp(-448, 448).to(FP8), (wu / 0.02).clamp(-448, 448).to(FP8)
        wd, sd = (wd / 0.01).clamp(-448, 448).to(FP8), torch.full((E, H // 128, I // 128), 0.01, device="cuda")
    x, topk, tw = (torch.empty((n, H), dtype=BF16, device="cuda"), torch.empty((n, K), dtype=torch.int32, device="cuda"),
                   torch.empty((n, K), device="cuda"))

    def step(group, x, topk, tw, a, y, out):
        h = ep.ep_create_handle(group, topk)
        ep.ep_dispatch(h, x)
        rows = ep.ep_handle_get_buffer(h, A.EP_BUF_LL_RECV)
        ep.ep_expert_gated(h, rows, wg, wu, a, **sc)
        if form == "fp8":
            q = torch.zeros((E * S * T, I), dtype=torch.uint8, device="cuda").view(FP8)
            qs = torch.zeros((E * S * T, I // 128), device="cuda")
            ep.ep_expert_quantize(h, a, q, qs)
            ep.ep_expert_linear(h, q, wd, y, x_scales=qs, w_scales=sd)
        else:
            ep.ep_expert_linear(h, a, wd, y)
        ep.ep_combine(h, y, tw, out)
        return h

    def buffers():
        return (torch.zeros((E, S * T, I), dtype=BF16, device="cuda"), torch.zeros((E, S * T, H), dtype=BF16, device="cuda"),
                torch.zeros((n, H), dtype=BF16, device="cuda"))

    def load(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn((n, H), generator=g, device="cuda"))
        topk.copy_(torch.argsort(torch.rand((n, E), generator=g, device="cuda"), dim=1)[:, :K])
        tw.copy_(torch.rand((n, K), generator=g, device="cuda"))
    load(0)
    gb, eb = buffers(), buffers()
    ep.ep_destroy_handle(step(one, x, topk, tw, *gb))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(one, x, topk, tw, *gb)
    for seed in range(1, 5):
        load(seed)
        graph.replay()
        torch.cuda.synchronize()
        ep.ep_destroy_handle(step(two, x, topk, tw, *eb))
        torch.cuda.synchronize()
        assert torch.equal(gb[2], eb[2]), seed
        assert bool(gb[2].isfinite().all())
    ep.ep_destroy_handle(held)
    ep.ep_destroy_group(one)
    ep.ep_destroy_group(two)
