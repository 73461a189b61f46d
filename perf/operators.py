"""The experts' products and the norms around the block: cases to measure, and their plain forms.

Operators (E experts, rows grouped by the routing handle; X[r] is a received row of expert e):
  gated       A[r] = act(X[r] Wg[e]^T) * (X[r] Wu[e]^T), and its backward pass;
  linear      Y[r] = X[r] W[e]^T (the down projection), and its backward pass;
  norm        x' = a*x + b*gate*rms(y; w_post) and rms(x'; w_pre), and its backward pass.

Where `own` is false, run() computes them with elementary torch operations in 32 bits, expert after
expert (a batched product would have to pad every expert to the fullest one, six times the work under the
routing study's scores); where it is true, it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _experts(name, op, mode, sources, tokens, experts, top_k, hidden, inter, form, act="silu", scores="uniform",
             grad="bf16"):
    return {"name": name, "op": op, "mode": mode, "sources": sources, "tokens": tokens, "experts": experts,
            "top_k": top_k, "hidden": hidden, "inter": inter, "form": form, "act": act, "scores": scores,
            "grad": grad}


def _norm(name, op, tokens, hidden, gate, post, weights):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "gate": gate, "post": post,
            "weights": weights}


def listed():
    return [
        # The smallest routing configuration (4 sources x 32 tokens, 16 experts, top-2): latency counts.
        _experts("gated_tiny", "gated", "ll", 4, 32, 16, 2, 256, 512, "bf16"),
        # Prefill of 4096 tokens, 256 experts, top-8, the routing study's skewed scores.
        _experts("gated_prefill_bf16", "gated", "ht", 1, 4096, 256, 8, 7168, 2048, "bf16", scores="page"),
        # The same in the serving form: dispatched FP8 rows, FP8 weights with one scale per 128 x 128 block.
        _experts("gated_prefill_fp8", "gated", "ht", 1, 4096, 256, 8, 7168, 2048, "fp8", scores="page"),
        # One decode step of one source's 128 tokens: the experts' weights are read for four rows each.
        _experts("gated_decode_fp8", "gated", "ll", 1, 128, 256, 8, 7168, 2048, "fp8"),
        # A training step's backward on a ragged batch: odd tokens, sizes that no tile divides, GELU.
        _experts("gated_backward_ragged", "gated_backward", "ht", 3, 333, 24, 3, 1040, 712, "bf16", act="gelu_tanh"),
        # A training step's backward on 4096 tokens, 64 experts, top-8.
        _experts("gated_backward_prefill", "gated_backward", "ht", 1, 4096, 64, 8, 7168, 2048, "bf16"),
        # Down projection of a decode step, FP8 activations and weights.
        _experts("linear_decode_fp8", "linear", "ll", 4, 16, 64, 8, 7168, 2048, "fp8"),
        # Down projection of the prefill.
        _experts("linear_prefill_bf16", "linear", "ht", 1, 4096, 256, 8, 7168, 2048, "bf16", scores="page"),
        # Its backward on 2048 tokens, the weights' gradients kept in 32 bits.
        _experts("linear_backward", "linear_backward", "ht", 1, 2048, 64, 8, 7168, 2048, "bf16", grad="f32"),
        # The norms around the block: one decode step, a prefill, and a training step's backward.
        _norm("norm_decode", "norm", 128, 7168, "none", False, "bf16"),
        _norm("norm_prefill", "norm", 16384, 7168, "channel", True, "f32"),
        _norm("norm_backward", "norm_backward", 4096, 7168, "channel", True, "f32"),
    ]


def _log(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "linear", "linear", "linear_backward", "norm", "norm_backward"])
    if op.startswith("norm"):
        case = _norm("", op, _log(rng, 1, 8192), _log(rng, 128, 8192, 16), rng.choice(["none", "channel", "token"]),
                     rng.random() < 0.6, rng.choice(["f32", "bf16"]))
        case.pop("name")
        return case
    form = "bf16" if "backward" in op else rng.choice(["bf16", "fp8"])
    mode = rng.choice(["ht", "ht", "ll"])
    experts = rng.choice([8, 16, 24, 64, 128])
    sources = rng.choice([1, 1, 2, 4])
    tokens = max(1, _log(rng, 1, 4096 if mode == "ht" else 256) // sources)
    step = 128 if form == "fp8" else 16
    case = _experts("", op, mode, sources, tokens, experts, rng.choice([1, 2, 6, 8]),
                    _log(rng, 256, 7168, step), _log(rng, 128, 2048, 128 if form == "fp8" else 8), form,
                    act=rng.choice(["silu", "gelu_tanh"]), scores=rng.choice(["uniform", "page"]),
                    grad=rng.choice(["bf16", "f32"]) if op == "linear_backward" else "bf16")
    case.pop("name")
    return case


# ---------------------------------------------------------------------------
# Routing: which rows the experts hold
# ---------------------------------------------------------------------------

def _topk(case, seed):
    """[n, K] distinct experts per token, drawn on the host: uniform scores, or the routing study's (a bias per expert)."""
    g = np.random.default_rng(seed)
    n, E = case["sources"] * case["tokens"], case["experts"]
    s = g.random((n, E), dtype=np.float32)
    if case["scores"] == "page":
        s += 0.5 * g.random(E, dtype=np.float32)
    return np.argsort(-s, axis=1, kind="stable")[:, :case["top_k"]].astype(np.int32)


def _rows(case, topk):
    """Rows of the receive layout in use, grouped by expert; rows per expert; rows the buffer has."""
    E, S, T = case["experts"], case["sources"], case["tokens"]
    counts = np.bincount(topk.reshape(-1), minlength=E)
    if case["mode"] == "ht":
        return np.arange(topk.size), counts, topk.size
    src = np.repeat(np.arange(S * T) // T, topk.shape[1])
    per = np.zeros((E, S), np.int64)
    np.add.at(per, (topk.reshape(-1), src), 1)
    slot = np.arange(T)[None, None, :] < per[:, :, None]     # [E, S, T] slots filled from the front
    return np.flatnonzero(slot.reshape(-1)), counts, E * S * T


class _Plan:
    """The library's group and handle of one routing, freed with the state."""

    def __init__(self, case, topk):
        import combine_ep_route_amd as ep
        self.ep = ep
        hidden = case["hidden"]
        kw = dict(mode="ht", num_nodes=1, ranks_per_node=1, num_experts=1, top_k=1, max_nodes_per_token=0,
                  hidden=hidden, max_tokens_per_rank=1, num_src_ranks=1, payload="bf16")
        if topk is not None:
            kw.update(mode=case["mode"], ranks_per_node=math.gcd(case["experts"], 8), num_experts=case["experts"],
                      top_k=case["top_k"], max_tokens_per_rank=case["tokens"], num_src_ranks=case["sources"],
                      payload=case["form"], ll_buffers=1, max_handles=1)
        self.group = ep.ep_create_group(**kw)
        self.handle = ep.ep_create_handle(self.group, topk) if topk is not None else None

    def __del__(self):
        if getattr(self, "group", None) is not None:
            self.ep.ep_destroy_group(self.group)
            self.group = None


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(shape, gen, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype) * scale


def _weights(E, N, K, gen):
    """[E, N, K] of standard deviation K^-1/2."""
    w = torch.empty((E, N, K), dtype=BF16, device="cuda")
    for e in range(E):
        w[e] = _randn((N, K), gen, BF16, K ** -0.5)
    return w


def _weights_fp8(E, N, K, gen):
    """The same in E4M3 with one fp32 scale per 128 x 128 block (the block's largest value becomes 448)."""
    q = torch.empty((E, N, K), dtype=FP8, device="cuda")
    s = torch.empty((E, N // 128, K // 128), dtype=torch.float32, device="cuda")
    for e in range(E):
        w = _randn((N, K), gen, scale=K ** -0.5).view(N // 128, 128, K // 128, 128)
        s[e] = w.abs().amax((1, 3)) / 448
        q[e] = (w / s[e][:, None, :, None]).reshape(N, K).to(FP8)
    return q, s


def _quantized(x):
    """E4M3 codes and one fp32 scale per 128 elements of each row."""
    b = x.float().view(x.shape[0], -1, 128)
    s = b.abs().amax(2) / 448
    return (b / s[:, :, None]).reshape(x.shape).to(FP8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, H = case["op"], case["hidden"]
    st = {"case": case}
    if op.startswith("norm"):
        n = case["tokens"]
        wt = torch.float32 if case["weights"] == "f32" else BF16
        st["y"] = _randn((n, H), gen, BF16, 0.7)
        st["x"] = _randn((n, H), gen, BF16, 2.0)
        st["w_pre"] = (1 + _randn((H,), gen, scale=0.2)).to(wt)
        st["w_post"] = (1 + _randn((H,), gen, scale=0.2)).to(wt) if case["post"] else None
        st["gate"] = None if case["gate"] == "none" else _randn((1 if case["gate"] == "channel" else n, H), gen, BF16, 0.5)
        st["g_res"] = _randn((n, H), gen, BF16)
        st["g_norm"] = _randn((n, H), gen, BF16)
        st["a"], st["b"], st["eps"] = 0.9, 0.6, 1e-6
        st["out_res"], st["out_norm"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        if own:
            st["plan"] = plan = _Plan(case, None)
            if op == "norm_backward":
                st["work"] = torch.empty(plan.ep.ep_residual_norm_workspace(plan.group, n), dtype=torch.uint8, device="cuda")
                st["g_y"] = torch.empty_like(st["y"])
                st["g_w"] = torch.empty((3, H), dtype=torch.float32, device="cuda")
                st["g_gate"] = torch.empty_like(st["gate"]) if case["gate"] == "token" else None
        return st
    E, I = case["experts"], case["inter"]
    K, N = (H, I) if op.startswith("gated") else (I, H)      # contracted size, columns of the output
    topk = _topk(case, seed)
    index, counts, rows = _rows(case, topk)
    st["index"] = torch.from_numpy(index).cuda()
    st["ends"] = [0] + np.cumsum(counts).tolist()
    # Rows in use hold values; the others are left as zeros.
    x = torch.zeros((rows, K), dtype=BF16, device="cuda")
    x[st["index"]] = _randn((len(index), K), gen, BF16)
    if case["form"] == "fp8":
        q, s = _quantized(x[st["index"]])
        if op == "gated":      # as the dispatch packs them: codes, then scales, rows on 128-byte boundaries
            used = K + K // 32
            st["x"] = torch.zeros((rows, -(-used // 128) * 128), dtype=torch.uint8, device="cuda")[:, :used]
            st["x"][st["index"]] = torch.cat([q.view(torch.uint8), s.view(torch.uint8)], 1)
        else:
            st["x"] = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
            st["x"][st["index"]] = q.view(torch.uint8)
            st["x"] = st["x"].view(FP8)
            st["x_scales"] = torch.zeros((rows, K // 128), dtype=torch.float32, device="cuda")
            st["x_scales"][st["index"]] = s
        st["w"], st["w_scales"] = _weights_fp8(E, N, K, gen)
        if op == "gated":
            st["w2"], st["w2_scales"] = _weights_fp8(E, N, K, gen)
    else:
        st["x"] = x
        st["w"] = _weights(E, N, K, gen)
        if op.startswith("gated"):
            st["w2"] = _weights(E, N, K, gen)
    if "backward" in op:
        st["g_out"] = torch.zeros((rows, N), dtype=BF16, device="cuda")
        st["g_out"][st["index"]] = _randn((len(index), N), gen, BF16)
        st["g_x"] = torch.zeros((rows, K), dtype=BF16, device="cuda")
        wt = torch.float32 if case["grad"] == "f32" else BF16
        st["g_w"] = torch.empty((E, N, K), dtype=wt, device="cuda")
        if op.startswith("gated"):
            st["g_w2"] = torch.empty((E, N, K), dtype=wt, device="cuda")
            st["g_gate"], st["g_up"] = torch.zeros_like(st["g_out"]), torch.zeros_like(st["g_out"])
    else:
        st["out"] = torch.zeros((rows, N), dtype=BF16, device="cuda")
    if own:
        st["plan"] = _Plan(case, torch.from_numpy(topk).cuda())
    return st


# ---------------------------------------------------------------------------
# One pass: the library's calls
# ---------------------------------------------------------------------------

def _own(st):
    case, plan = st["case"], st["plan"]
    ep, op = plan.ep, case["op"]
    if op == "gated":
        ep.ep_expert_gated(plan.handle, st["x"], st["w"], st["w2"], st["out"], activation=case["act"],
                           w_gate_scales=st.get("w_scales"), w_up_scales=st.get("w2_scales"))
        return st["out"]
    if op == "gated_backward":
        ep.ep_expert_gated_backward(plan.handle, st["x"], st["w"], st["w2"], st["g_out"], st["g_gate"], st["g_up"],
                                    activation=case["act"], grad_rows=st["g_x"], grad_w_gate=st["g_w"],
                                    grad_w_up=st["g_w2"])
        return {"x": st["g_x"], "gate": st["g_gate"], "up": st["g_up"], "w_gate": st["g_w"], "w_up": st["g_w2"]}
    if op == "linear":
        ep.ep_expert_linear(plan.handle, st["x"], st["w"], st["out"], x_scales=st.get("x_scales"),
                            w_scales=st.get("w_scales"))
        return st["out"]
    if op == "linear_backward":
        ep.ep_expert_linear_backward(plan.handle, st["x"], st["w"], st["g_out"], grad_x=st["g_x"], grad_w=st["g_w"])
        return {"x": st["g_x"], "w": st["g_w"]}
    if op == "norm":
        ep.ep_residual_norm(plan.group, st["y"], st["x"], st["out_res"], st["out_norm"], st["w_pre"],
                            w_post=st["w_post"], gate=st["gate"], residual_scale=st["a"], block_scale=st["b"],
                            eps=st["eps"])
        return {"residual": st["out_res"], "norm": st["out_norm"]}
    gate = case["gate"]
    ep.ep_residual_norm_backward(plan.group, st["y"], st["x"], st["g_res"], st["g_norm"], st["w_pre"], st["out_res"],
                                 st["g_y"], st["g_w"][0], st["work"], w_post=st["w_post"], gate=st["gate"],
                                 grad_w_post=st["g_w"][1] if case["post"] else None,
                                 grad_gate=None if gate == "none" else st["g_w"][2:3] if gate == "channel" else st["g_gate"],
                                 residual_scale=st["a"], block_scale=st["b"], eps=st["eps"])
    got = {"residual": st["out_res"], "y": st["g_y"], "w_pre": st["g_w"][0]}
    if case["post"]:
        got["w_post"] = st["g_w"][1]
    if gate != "none":
        got["gate"] = st["g_w"][2:3] if gate == "channel" else st["g_gate"]
    return got


# ---------------------------------------------------------------------------
# One pass: the plain form
# ---------------------------------------------------------------------------

def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _x32(st):
    """The rows in use, in 32 bits."""
    case, x = st["case"], st["x"][st["index"]]
    if case["form"] != "fp8":
        return x.float()
    if case["op"] == "gated":
        H = case["hidden"]
        q, s = x[:, :H].contiguous().view(FP8), x[:, H:].contiguous().view(torch.float32)
    else:
        q, s = x, st["x_scales"][st["index"]]
    return (q.float().view(q.shape[0], -1, 128) * s[:, :, None]).view(q.shape)


def _w32(st, name, e):
    w = st[name][e].float()
    if st["case"]["form"] != "fp8":
        return w
    N, K = w.shape
    return (w.view(N // 128, 128, K // 128, 128) * st[name + "_scales"][e][:, None, :, None]).view(N, K)


def _plain_experts(st):
    case = st["case"]
    op, index, ends = case["op"], st["index"], st["ends"]
    x = _x32(st)
    if "backward" in op:
        g = st["g_out"][index].float()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            if "backward" in op:
                st["g_w"][e] = 0
                if op == "gated_backward":
                    st["g_w2"][e] = 0
            continue
        at, xe, w = index[a:b], x[a:b], _w32(st, "w", e)
        if op == "linear":
            st["out"][at] = (xe @ w.t()).to(BF16)
        elif op == "linear_backward":
            st["g_x"][at] = (g[a:b] @ w).to(BF16)
            st["g_w"][e] = g[a:b].t() @ xe
        else:
            w2 = _w32(st, "w2", e)
            pre, up = xe @ w.t(), xe @ w2.t()
            act, slope = _act(pre, case["act"])
            if op == "gated":
                st["out"][at] = (act * up).to(BF16)
            else:
                d_pre, d_up = g[a:b] * up * slope, g[a:b] * act
                st["g_gate"][at], st["g_up"][at] = d_pre.to(BF16), d_up.to(BF16)
                st["g_x"][at] = (d_pre @ w + d_up @ w2).to(BF16)
                st["g_w"][e], st["g_w2"][e] = d_pre.t() @ xe, d_up.t() @ xe
    if op == "gated_backward":
        return {"x": st["g_x"], "gate": st["g_gate"], "up": st["g_up"], "w_gate": st["g_w"], "w_up": st["g_w2"]}
    return {"x": st["g_x"], "w": st["g_w"]} if op == "linear_backward" else st["out"]


def _rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(1, keepdim=True) + eps)


def _plain_norm(st):
    case, a, b, eps = st["case"], st["a"], st["b"], st["eps"]
    y, x, w_pre = st["y"].float(), st["x"].float(), st["w_pre"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    w_post = st["w_post"].float() if case["post"] else None
    r_y = _rms(y, eps) if case["post"] else None
    t = y * r_y * w_post if case["post"] else y
    if case["op"] == "norm":
        res = (a * x + b * gate * t).to(BF16)
        z = res.float()                                     # the next norm reads the stream as it is kept
        return {"residual": res, "norm": (z * _rms(z, eps) * w_pre).to(BF16)}
    g_res, g_norm = st["g_res"].float(), st["g_norm"].float()
    r = _rms(x, eps)
    wg = g_norm * w_pre
    dx = g_res + r * wg - x * (r * r * r) * (wg * x).mean(1, keepdim=True)
    dt = b * gate * dx
    got = {"residual": (a * dx).to(BF16), "w_pre": (g_norm * x * r).sum(0)}
    if case["post"]:
        wt = dt * w_post
        got["y"] = (r_y * wt - y * (r_y * r_y * r_y) * (wt * y).mean(1, keepdim=True)).to(BF16)
        got["w_post"] = (dt * y * r_y).sum(0)
    else:
        got["y"] = dt.to(BF16)
    if case["gate"] == "channel":
        got["gate"] = (b * dx * t).sum(0, keepdim=True)
    elif case["gate"] == "token":
        got["gate"] = (b * dx * t).to(BF16)
    return got


def run(st):
    if own:
        return _own(st)
    return _plain_norm(st) if st["case"]["op"].startswith("norm") else _plain_experts(st)


# ---------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, H = case["op"], case["hidden"]
    if op.startswith("norm"):
        n, token_gate = case["tokens"], case["gate"] == "token"
        tensors = (4 if op == "norm" else 6) + token_gate * (1 if op == "norm" else 2)
        return {"bytes": tensors * n * H * 2, "flops": (12 if op == "norm" else 30) * n * H}
    E, I = case["experts"], case["inter"]
    topk = _topk(case, 0)
    rows, active = topk.size, len(np.unique(topk))
    K, N = (H, I) if op.startswith("gated") else (I, H)
    mats = 2 if op.startswith("gated") else 1
    product = 2 * rows * K * N * mats
    if "backward" in op:
        grad = E * mats * N * K * (4 if case["grad"] == "f32" else 2)
        act = rows * (2 * K + N + (2 * N if mats == 2 else 0)) * 2
        return {"bytes": active * mats * N * K * 2 + grad + act, "flops": product * (3 if mats == 2 else 2)}
    size = 1 if case["form"] == "fp8" else 2
    extra = (rows * K // 32 + active * mats * (N // 128) * (K // 128) * 4) if size == 1 else 0
    return {"bytes": active * mats * N * K * size + rows * K * size + rows * N * 2 + extra, "flops": product}


def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    if case["op"].startswith("norm"):
        return _exact_norm(st, D)
    E, op, H = case["experts"], case["op"], case["hidden"]
    gated, backward = op.startswith("gated"), "backward" in op
    got = {}

    def values(name, e, at):
        if name == "x":
            x = st["x"][at]
            if case["form"] != "fp8":
                return x.to(D)
            if gated:
                q, s = x[:, :H].contiguous().view(FP8), x[:, H:].contiguous().view(torch.float32)
            else:
                q, s = x, st["x_scales"][at]
            return q.to(D) * torch.repeat_interleave(s.to(D), 128, dim=1)
        w = st[name][e].to(D)
        if case["form"] == "fp8":
            s = st[name + "_scales"][e].to(D)
            w = w * torch.repeat_interleave(torch.repeat_interleave(s, 128, dim=0), 128, dim=1)
        return w

    def like(t):
        return torch.zeros(t.shape, dtype=D, device="cuda")

    if backward:
        got["x"], got["w_gate" if gated else "w"] = like(st["g_x"]), like(st["g_w"])
        if gated:
            got["gate"], got["up"], got["w_up"] = like(st["g_gate"]), like(st["g_up"]), like(st["g_w2"])
    else:
        got = like(st["out"])
    for e in range(E):
        at = st["index"][st["ends"][e]:st["ends"][e + 1]]
        if len(at) == 0:
            continue
        x, w = values("x", e, at), values("w", e, at)
        if not gated and not backward:
            got[at] = torch.mm(x, w.t())
            continue
        g = st["g_out"][at].to(D) if backward else None
        if not gated:
            got["x"][at], got["w"][e] = torch.mm(g, w), torch.mm(g.t(), x)
            continue
        w2 = values("w2", e, at)
        p = torch.mm(x, w.t())
        u = torch.mm(x, w2.t())
        if case["act"] == "silu":
            sig = torch.sigmoid(p)
            f, df = p * sig, sig + p * sig * (1 - sig)
        else:                                # 0.5 p (1 + tanh z) = p * sigmoid(2z)
            c = math.sqrt(8 / math.pi)
            sig = torch.sigmoid(c * (p + 0.044715 * p ** 3))
            f, df = p * sig, sig + p * sig * (1 - sig) * c * (1 + 0.134145 * p ** 2)
        if not backward:
            got[at] = f * u
            continue
        dp, du = g * u * df, g * f
        got["gate"][at], got["up"][at] = dp, du
        got["x"][at] = torch.mm(dp, w) + torch.mm(du, w2)
        got["w_gate"][e], got["w_up"][e] = torch.mm(dp.t(), x), torch.mm(du.t(), x)
    return got


def _exact_norm(st, D):
    case, a, b, eps = st["case"], st["a"], st["b"], st["eps"]
    y, x, wn = st["y"].to(D), st["x"].to(D), st["w_pre"].to(D)
    gate = torch.ones((1, 1), dtype=D, device="cuda") if st["gate"] is None else st["gate"].to(D)

    def hat(v):
        return v / torch.sqrt(v.square().mean(dim=1, keepdim=True) + eps)

    def back(v, g):      # adjoint of hat at v
        s = torch.sqrt(v.square().mean(dim=1, keepdim=True) + eps)
        return (g - hat(v) * (g * hat(v)).mean(dim=1, keepdim=True)) / s

    wp = st["w_post"].to(D) if case["post"] else None
    block = hat(y) * wp if case["post"] else y
    if case["op"] == "norm":
        z = a * x + gate * block * b
        return {"residual": z, "norm": hat(z) * wn}
    gn = st["g_norm"].to(D)
    dx = st["g_res"].to(D) + back(x, gn * wn)
    dt = dx * gate * b
    got = {"residual": dx * a, "w_pre": (gn * hat(x)).sum(dim=0), "y": back(y, dt * wp) if case["post"] else dt}
    if case["post"]:
        got["w_post"] = (dt * hat(y)).sum(dim=0)
    if case["gate"] != "none":
        d = dx * block * b
        got["gate"] = d.sum(dim=0, keepdim=True) if case["gate"] == "channel" else d
    return got
