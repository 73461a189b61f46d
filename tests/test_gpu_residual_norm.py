"""ep_residual_norm and its backward pass against 64-bit references.

Bounds, per element.  An fp32 sum of H terms of one sign is within H 2^-24 of itself, a general one within
H 2^-24 of the sum of the terms' magnitudes; a norm's factor is then within H 2^-24 of itself, and the
dozen other roundings of a value add 2^-24 of its terms' magnitudes each: (H + 32) 2^-23 of the
magnitudes covers both (n more terms for a sum over n rows), and a rounding to bf16 2^-8 of the value.
"""
import pytest
import torch

from expert_util import BF16, D, HALF, near, normal
from gpu_util import ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture
def group():
    made = []

    def make(H):
        made.append(ep.ep_create_group(mode="ht", num_nodes=1, ranks_per_node=1, num_experts=1, top_k=1,
                                       max_nodes_per_token=0, hidden=H, max_tokens_per_rank=1, num_src_ranks=1,
                                       payload="bf16"))
        return made[-1]
    yield make
    for g in made:
        ep.ep_destroy_group(g)


def padded(t, pad):
    """The same values in rows that are `pad` elements further apart."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def inputs(n, H, gate, post, wtype, pad):
    x, y = padded(normal((n, H), 1, 2.0), pad), padded(normal((n, H), 2, 0.7), 2 * pad)
    wn = (1 + normal((H,), 3, 0.2, torch.float32)).to(wtype)
    wp = (1 + normal((H,), 4, 0.2, torch.float32)).to(wtype) if post else None
    g = None if gate == "none" else padded(normal((1 if gate == "channel" else n, H), 5, 0.5), pad)
    return x, y, wn, wp, g


def rms(v, eps):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


CASES = [(1, 16, "none", False, BF16, 0), (1, 7168, "token", True, torch.float32, 0),
         (5, 272, "channel", True, BF16, 8), (130, 1040, "token", False, torch.float32, 16),
         (1, 512, "channel", False, BF16, 0), (600, 2048, "channel", True, torch.float32, 8),
         (3, 8192, "none", True, BF16, 0), (7, 8208, "channel", True, torch.float32, 8),
         (2, 16384, "token", True, BF16, 0), (33, 14352, "none", False, torch.float32, 0)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, group):
    n, H, gate, post, wtype, pad = case
    say(f"residual norm {case}")
    x, y, wn, wp, g = inputs(*case)
    a, b, eps = 0.9, -0.6, 1e-5
    res = padded(torch.zeros((n, H), dtype=BF16, device="cuda"), pad)
    out = padded(torch.zeros((n, H), dtype=BF16, device="cuda"), 3 * pad)
    ep.ep_residual_norm(group(H), y, x, res, out, wn, w_post=wp, gate=g, residual_scale=a, block_scale=b, eps=eps)
    t = y.to(D)
    if post:
        t = t * rms(t, eps) * wp.to(D)
    if g is not None:
        t = t * g.to(D)
    a32, b32 = float(torch.tensor(a, dtype=torch.float32)), float(torch.tensor(b, dtype=torch.float32))
    want = a32 * x.to(D) + b32 * t
    slack = (H + 32) * 2.0 ** -23
    near(res, want, slack * (abs(a) * x.to(D).abs() + abs(b) * t.abs()) * 1.01 + HALF * want.abs() * 1.01, "stream")
    z = res.to(D)
    v = z * rms(z, eps) * wn.to(D)
    near(out, v, (slack + HALF * 1.01) * v.abs(), "norm")


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("with_res", [True, False], ids=["stream_grad", "no_stream_grad"])
def test_backward(case, with_res, group):
    n, H, gate, post, wtype, pad = case
    say(f"residual norm backward {case} {with_res}")
    x, y, wn, wp, g = inputs(*case)
    a, b, eps = 0.9, -0.6, 1e-5
    gr = padded(normal((n, H), 6), pad) if with_res else None
    gn = padded(normal((n, H), 7), pad)
    dres, dy = torch.zeros((n, H), dtype=BF16, device="cuda"), torch.zeros((n, H), dtype=BF16, device="cuda")
    sums = torch.full((3, H), 5.0, device="cuda")
    dgate = None if gate == "none" else sums[2:3] if gate == "channel" else torch.zeros((n, H), dtype=BF16, device="cuda")
    gp = group(H)
    work = torch.full((ep.ep_residual_norm_workspace(gp, n),), 255, dtype=torch.uint8, device="cuda")
    ep.ep_residual_norm_backward(gp, y, x, gr, gn, wn, dres, dy, sums[0], work, w_post=wp, gate=g,
                                 grad_w_post=sums[1] if post else None, grad_gate=dgate, residual_scale=a,
                                 block_scale=b, eps=eps)
    a, b = (float(torch.tensor(v, dtype=torch.float32)) for v in (a, b))
    X, Y, GN = x.to(D), y.to(D), gn.to(D)
    leaves = [t.to(D).requires_grad_() for t in (X, Y, wn)] + \
        [t.to(D).requires_grad_() if t is not None else None for t in (wp, g)]
    lx, ly, lwn, lwp, lg = leaves
    # gradients of the formula: the norm at x, and the block's part of the stream
    (lx * rms(lx, eps) * lwn).backward(GN)
    dx = lx.grad + (gr.to(D) if with_res else 0)
    t = ly * rms(ly, eps) * lwp if post else ly * 1
    (b * (t if lg is None else t * lg)).backward(dx)
    slack = (H + n + 32) * 2.0 ** -23 * 1.1
    r = rms(X, eps)
    vm = (GN * wn.to(D)).abs()
    mag = (gr.to(D).abs() if with_res else 0) + r * (vm + (X * r).abs() * (vm * (X * r).abs()).mean(1, keepdim=True))
    near(dres, a * dx, slack * abs(a) * mag + HALF * 1.01 * (a * dx).abs(), "residual")
    near(sums[0], lwn.grad, slack * (GN * X * r).abs().sum(0) + 1e-30, "w_pre")
    gm = 1 if g is None else g.to(D).abs()
    dtm = abs(b) * gm * mag
    if post:
        ry = rms(Y, eps)
        q = dtm * wp.to(D).abs()
        ym = ry * (q + (Y * ry).abs() * (q * (Y * ry).abs()).mean(1, keepdim=True))
        near(sums[1], lwp.grad, slack * (dtm * (Y * ry).abs()).sum(0) + 1e-30, "w_post")
        tm = (Y * ry * wp.to(D)).abs()
    else:
        ym, tm = dtm, Y.abs()
    near(dy, ly.grad, slack * ym + HALF * 1.01 * ly.grad.abs(), "y")
    if gate == "channel":
        near(dgate, lg.grad, slack * (abs(b) * mag * tm).sum(0, keepdim=True) + 1e-30, "gate")
    elif gate == "token":
        near(dgate, lg.grad, slack * abs(b) * mag * tm + HALF * 1.01 * lg.grad.abs(), "gate")
    if not post:
        assert bool((sums[1] == 5.0).all())


def test_in_place_and_repeated(group):
    """out_residual in place of residual, out_norm in place of y; the same for the gradients; the same bits twice."""
    say("residual norm in place")
    n, H = 77, 1040
    gp = group(H)
    x, y, wn, wp, g = inputs(n, H, "channel", True, BF16, 0)
    kw = dict(w_post=wp, gate=g, residual_scale=0.5, block_scale=2.0)
    res, out = torch.empty_like(x), torch.empty_like(x)
    ep.ep_residual_norm(gp, y, x, res, out, wn, **kw)
    x2, y2 = x.clone(), y.clone()
    ep.ep_residual_norm(gp, y2, x2, x2, y2, wn, **kw)
    assert torch.equal(x2, res) and torch.equal(y2, out)

    gr, gn = normal((n, H), 6), normal((n, H), 7)
    work = torch.empty(ep.ep_residual_norm_workspace(gp, n), dtype=torch.uint8, device="cuda")
    first = None
    for place in ("apart", "y", "norm"):
        a, c, d = gr.clone(), gn.clone(), y.clone()
        dres, dy = (torch.empty_like(x), torch.empty_like(x)) if place == "apart" else (a, d if place == "y" else c)
        sums = torch.empty((3, H), device="cuda")
        ep.ep_residual_norm_backward(gp, d, x, a, c, wn, dres, dy, sums[0], work, grad_w_post=sums[1],
                                     grad_gate=sums[2:3], **kw)
        got = [t.clone() for t in (dres, dy, sums)]
        first = first or got
        assert all(torch.equal(p, q) for p, q in zip(first, got)), place


def test_no_rows(group):
    say("residual norm of no rows")
    gp = group(256)
    e = torch.empty((0, 256), dtype=BF16, device="cuda")
    w = torch.ones(256, device="cuda")
    ep.ep_residual_norm(gp, e, e, e, e, w, w_post=w)
    sums = torch.full((3, 256), 5.0, device="cuda")
    ep.ep_residual_norm_backward(gp, e, e, e, e, w, e, e, sums[0], torch.empty(0, dtype=torch.uint8, device="cuda"),
                                 w_post=w, gate=torch.ones((1, 256), dtype=BF16, device="cuda"), grad_w_post=sums[1],
                                 grad_gate=sums[2:3])
    assert bool((sums == 0).all())


@pytest.mark.parametrize("what", ["forward", "backward"])
def test_zero_rows_and_far_values(group, what):
    """A row of zeros gives a norm of zeros (eps alone under the root), and values that are not finite stay in their row."""
    say(f"residual norm {what}: zero row, infinity, NaN")
    gp = group(512)
    x, y, wn, _, _ = inputs(4, 512, "none", False, torch.float32, 0)
    x[0], y[0] = 0, 0
    y[1, 3], x[2, 5] = float("inf"), float("nan")
    work = torch.empty(ep.ep_residual_norm_workspace(gp, 4), dtype=torch.uint8, device="cuda")
    res, out = torch.empty_like(x), torch.empty_like(x)
    if what == "forward":
        ep.ep_residual_norm(gp, y, x, res, out, wn)
        assert bool((res[0] == 0).all()) and bool((out[0] == 0).all())
    else:
        ep.ep_residual_norm_backward(gp, y, x, None, normal((4, 512), 7), wn, res, out, torch.empty(512, device="cuda"),
                                     work)
        assert bool(res[0].isfinite().all()) and bool(out[0].isfinite().all())
    assert bool(res[3].isfinite().all()) and bool(out[3].isfinite().all())
    assert not bool(out[2].isfinite().all())
