"""Rows of ranks in expert order and back, and backward passes from rows kept in 8 bits: cases to measure, and plain forms.

Operators (the per-rank layout leaves one row per token and destination rank; `row(i, k)` is the rank's row of entry k of
token i, `place(i, k)` the entry's place in expert order):
  sort             S[place(i,k)] = X[row(i,k)], packed FP8 rows or BF16 ones;
  sort_backward    dX[r] = sum of dS[place(i,k)] over the entries with row(i,k) = r;
  unsort           P[r] = sum of w[i,k] Y[place(i,k)] over them;
  unsort_backward  dY[place(i,k)] = w[i,k] dP[row(i,k)], dw[i,k] = <dP[row(i,k)], Y[place(i,k)]>;
  gated_backward   of A = act(X Wg^T) * (X Wu^T) from E4M3 rows X with a scale per 128 values;
  linear_backward  of Y = X W^T from such rows.

Where `own` is false, run() computes them with elementary torch operations in 32 bits (the products expert after expert: a
batched product would have to pad every expert to the fullest one); where it is true, it makes the library's calls.
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

def _move(name, op, nodes, ranks, sources, tokens, experts, top_k, hidden, form="bf16", scores="uniform"):
    """A move between the rows of nodes x ranks ranks and the experts' order; up to half of the nodes a token."""
    return {"name": name, "op": op, "nodes": nodes, "ranks": ranks, "sources": sources, "tokens": tokens,
            "experts": experts, "top_k": top_k, "hidden": hidden, "form": form, "scores": scores}


def _product(name, op, mode, sources, tokens, experts, top_k, hidden, inter, act="silu", scores="uniform"):
    return {"name": name, "op": op, "mode": mode, "sources": sources, "tokens": tokens, "experts": experts,
            "top_k": top_k, "hidden": hidden, "inter": inter, "act": act, "scores": scores}


def listed():
    return [
        # The smallest routing configuration (4 sources x 32 tokens, 4 ranks, 16 experts, top-2): latency counts.
        _move("sort_tiny", "sort", 2, 2, 4, 32, 16, 2, 256),
        # Prefill of 4096 tokens over 8 x 8 ranks, the dispatch's packed FP8 rows.
        _move("sort_prefill_fp8", "sort", 8, 8, 1, 4096, 256, 8, 7168, form="fp8", scores="page"),
        # A training step's backward on a ragged batch: odd tokens, a row size that no tile divides.
        _move("sort_backward_ragged", "sort_backward", 2, 2, 3, 333, 24, 3, 1040),
        # The backward of 16384 tokens.
        _move("sort_backward_long", "sort_backward", 8, 8, 1, 16384, 256, 8, 7168),
        # A small batch's way back: one source's 128 tokens.
        _move("unsort_small", "unsort", 8, 8, 1, 128, 256, 8, 7168),
        # The prefill's way back.
        _move("unsort_prefill", "unsort", 8, 8, 1, 4096, 256, 8, 7168, scores="page"),
        # Their gradients, the routing weights' among them: few ranks, so that many entries share a row; the prefill's.
        _move("unsort_backward_shared", "unsort_backward", 2, 2, 2, 500, 64, 6, 2048),
        _move("unsort_backward_prefill", "unsort_backward", 8, 8, 1, 4096, 256, 8, 7168, scores="page"),
        # A training step of a ragged batch from the dispatched FP8 rows: odd tokens, tanh GELU.
        _product("gated_backward_ragged", "gated_backward", "ht", 3, 333, 24, 3, 1152, 712, act="gelu_tanh"),
        # A training step of 4096 tokens, 64 experts, top-8.
        _product("gated_backward_prefill", "gated_backward", "ht", 1, 4096, 64, 8, 7168, 2048),
        # The down projection's backward from quantised activations: 4 sources' slots, 16 rows an expert.
        _product("linear_backward_slots", "linear_backward", "ll", 4, 64, 64, 4, 1024, 768),
        # The same of a training step of 4096 tokens.
        _product("linear_backward_prefill", "linear_backward", "ht", 1, 4096, 64, 8, 7168, 2048, scores="page"),
    ]


def _log(rng, low, high, step=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step))


def draw(rng):
    op = rng.choice(["sort", "sort", "sort_backward", "unsort", "unsort", "unsort_backward", "gated_backward",
                     "linear_backward"])
    if op in ("gated_backward", "linear_backward"):
        mode = rng.choice(["ht", "ht", "ll"])
        sources = rng.choice([1, 1, 2, 3, 4])
        tokens = max(1, _log(rng, 1, 4096 if mode == "ht" else 256) // sources)
        down = op == "linear_backward"      # its rows have `inter` columns, the gated product's `hidden` ones
        case = _product("", op, mode, sources, tokens, rng.choice([8, 16, 24, 40, 64]), rng.choice([1, 2, 3, 6, 8]),
                        _log(rng, 256, 7168, 16 if down else 128), _log(rng, 128, 2048, 128 if down else 8),
                        act=rng.choice(["silu", "gelu_tanh"]), scores=rng.choice(["uniform", "page"]))
    else:
        nodes, ranks, experts = rng.choice([(1, 2, 8), (2, 2, 16), (2, 2, 24), (2, 4, 64), (4, 8, 128), (8, 8, 256)])
        sources = min(nodes * ranks, rng.choice([1, 1, 2, 3, 4]))
        form = rng.choice(["bf16", "fp8"]) if op == "sort" else "bf16"
        case = _move("", op, nodes, ranks, sources, max(1, _log(rng, 1, 8192) // sources), experts,
                     rng.choice([1, 2, 3, 6, 8]), _log(rng, 128, 7168, 128 if form == "fp8" else 16), form=form,
                     scores=rng.choice(["uniform", "page"]))
    case.pop("name")
    return case


# ---------------------------------------------------------------------------
# Routing: who holds which rows
# ---------------------------------------------------------------------------

def _topk(case, seed):
    """[n, K] distinct experts per token, drawn on the host: uniform scores, or the routing study's (a bias per expert).
    Over several nodes a token keeps the better half of them, by the sum of each node's two best scores."""
    g = np.random.default_rng(seed)
    n, E, K = case["sources"] * case["tokens"], case["experts"], case["top_k"]
    s = g.random((n, E), dtype=np.float32)
    if case["scores"] == "page":
        s += 0.5 * g.random(E, dtype=np.float32)
    N = case.get("nodes", 1)
    if N > 1 and E // N * (N // 2) >= K:
        best = np.sort(s.reshape(n, N, E // N), axis=2)[:, :, -2:].sum(2)
        away = np.argsort(best, axis=1)[:, :N - N // 2]
        np.put_along_axis(s.reshape(n, N, E // N), away[:, :, None], -1.0, axis=1)
    return np.argsort(-s, axis=1, kind="stable")[:, :K].astype(np.int32)


def _places(case, topk):
    """Of every place in expert order its entry (i * K + k) and its rank's row; the number of rank rows."""
    n, R = topk.shape[0], case["nodes"] * case["ranks"]
    flat = topk.reshape(-1)
    entry = np.argsort(flat, kind="stable")          # by expert, tokens ascending
    key = (flat // (case["experts"] // R)).astype(np.int64) * n + np.arange(flat.size) // topk.shape[1]
    used, row = np.unique(key, return_inverse=True)  # by rank, tokens ascending
    return entry, row[entry], used.size


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
        kw = dict(num_experts=case["experts"], top_k=case["top_k"], max_nodes_per_token=0, hidden=case["hidden"],
                  max_tokens_per_rank=case["tokens"], num_src_ranks=case["sources"], max_handles=1)
        if "mode" in case:
            kw.update(mode=case["mode"], num_nodes=1, ranks_per_node=math.gcd(case["experts"], 8), ll_buffers=1,
                      payload="fp8" if case["op"] == "gated_backward" else "bf16")
        else:
            kw.update(mode="ht", ht_stage2="rank_sorted", num_nodes=case["nodes"], ranks_per_node=case["ranks"],
                      payload=case["form"])
        self.group = ep.ep_create_group(**kw)
        self.handle = ep.ep_create_handle(self.group, topk)

    def __del__(self):
        if getattr(self, "group", None) is not None:
            self.ep.ep_destroy_group(self.group)
            self.group = None


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(shape, gen, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype) * scale


def _packed(rows, H):
    """U8 rows of H codes and their scales, on 128-byte boundaries as the dispatch packs them."""
    used = H + H // 32
    return torch.zeros((rows, -(-used // 128) * 128), dtype=torch.uint8, device="cuda")[:, :used]


def _quantized(x):
    """E4M3 codes and one fp32 scale per 128 elements of each row."""
    b = x.float().view(x.shape[0], -1, 128)
    s = b.abs().amax(2) / 448
    return (b / s[:, :, None]).reshape(x.shape).to(FP8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    topk = _topk(case, seed)
    st = {"case": case}
    if "mode" in case:
        _prepare_product(case, topk, gen, st)
    else:
        _prepare_move(case, topk, gen, st)
    if own:
        st["plan"] = _Plan(case, torch.from_numpy(topk).cuda())
    return st


def _prepare_move(case, topk, gen, st):
    op, H = case["op"], case["hidden"]
    entry, row, rows = _places(case, topk)
    st["entry"], st["row"] = torch.from_numpy(entry).cuda(), torch.from_numpy(row).cuda()
    places, st["rows"] = topk.size, rows
    if op == "sort":
        x = _randn((rows, H), gen, BF16)
        if case["form"] == "fp8":
            q, s = _quantized(x)
            st["x"], st["out"] = _packed(rows, H), _packed(places, H)
            st["x"].copy_(torch.cat([q.view(torch.uint8), s.view(torch.uint8)], 1))
        else:
            st["x"], st["out"] = x, torch.empty((places, H), dtype=BF16, device="cuda")
        return
    if op != "sort_backward":
        w = torch.softmax(_randn(topk.shape, gen, scale=1.0), 1)     # a token's weights sum to one
        st["w"] = w.contiguous()
    if op == "unsort_backward":
        st["g"] = _randn((rows, H), gen, BF16)
        st["g_y"] = torch.empty((places, H), dtype=BF16, device="cuda")
        st["g_w"] = torch.empty(topk.shape, dtype=torch.float32, device="cuda")
    else:
        # as many rows as a routing may need; those behind the last one in use are not written
        most = topk.shape[0] * min(case["top_k"], case["nodes"] * case["ranks"])
        st["out"] = torch.zeros((most, H), dtype=BF16, device="cuda")
    st["y"] = _randn((places, H), gen, BF16)


def _prepare_product(case, topk, gen, st):
    op, E = case["op"], case["experts"]
    K, N = (case["hidden"], case["inter"]) if op == "gated_backward" else (case["inter"], case["hidden"])
    index, counts, rows = _rows(case, topk)
    st["index"] = torch.from_numpy(index).cuda()
    st["ends"] = [0] + np.cumsum(counts).tolist()
    q, s = _quantized(_randn((len(index), K), gen, BF16))
    if op == "gated_backward":      # as the dispatch packs them: codes, then scales
        st["x"] = _packed(rows, K)
        st["x"][st["index"]] = torch.cat([q.view(torch.uint8), s.view(torch.uint8)], 1)
    else:
        st["x"] = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
        st["x"][st["index"]] = q.view(torch.uint8)
        st["x"] = st["x"].view(FP8)
        st["x_scales"] = torch.zeros((rows, K // 128), dtype=torch.float32, device="cuda")
        st["x_scales"][st["index"]] = s
    for name in ("w", "w2") if op == "gated_backward" else ("w",):
        st[name] = torch.empty((E, N, K), dtype=BF16, device="cuda")
        for e in range(E):
            st[name][e] = _randn((N, K), gen, BF16, K ** -0.5)
        st["g_" + name] = torch.empty_like(st[name])
    st["g_out"] = torch.zeros((rows, N), dtype=BF16, device="cuda")
    st["g_out"][st["index"]] = _randn((len(index), N), gen, BF16)
    st["g_x"] = torch.zeros((rows, K), dtype=BF16, device="cuda")
    if op == "gated_backward":
        st["g_gate"], st["g_up"] = torch.zeros_like(st["g_out"]), torch.zeros_like(st["g_out"])


# ---------------------------------------------------------------------------
# One pass: the library's calls
# ---------------------------------------------------------------------------

def _own(st):
    case, plan = st["case"], st["plan"]
    ep, op = plan.ep, case["op"]
    if op == "sort":
        ep.ep_expert_sort(plan.handle, st["x"], st["out"])
    elif op == "sort_backward":
        ep.ep_expert_sort_backward(plan.handle, st["y"], st["out"])
    elif op == "unsort":
        ep.ep_expert_unsort(plan.handle, st["y"], st["w"], st["out"])
    elif op == "unsort_backward":
        ep.ep_expert_unsort_backward(plan.handle, st["g"], st["w"], st["g_y"], expert_out=st["y"],
                                     grad_weights=st["g_w"])
    elif op == "gated_backward":
        ep.ep_expert_gated_backward_fp8(plan.handle, st["x"], st["w"], st["w2"], st["g_out"], st["g_gate"],
                                        st["g_up"], activation=case["act"], grad_rows=st["g_x"],
                                        grad_w_gate=st["g_w"], grad_w_up=st["g_w2"])
    else:
        ep.ep_expert_linear_backward_fp8(plan.handle, st["x"], st["x_scales"], st["w"], st["g_out"],
                                         grad_x=st["g_x"], grad_w=st["g_w"])


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


def _plain_move(st):
    case, row, entry = st["case"], st["row"], st["entry"]
    op = case["op"]
    if op == "sort":
        st["out"].copy_(st["x"][row])
    elif op == "unsort_backward":
        g, w = st["g"].float()[row], st["w"].view(-1)[entry]
        st["g_y"].copy_(g * w[:, None])
        st["g_w"].view(-1)[entry] = (g * st["y"].float()).sum(1)
    else:
        y = st["y"].float()
        if op == "unsort":
            y = y * st["w"].view(-1)[entry][:, None]
        total = torch.zeros((st["rows"], y.shape[1]), dtype=torch.float32, device="cuda")
        st["out"][:st["rows"]].copy_(total.index_add_(0, row, y))


def _plain_product(st):
    case, index, ends = st["case"], st["index"], st["ends"]
    gated = case["op"] == "gated_backward"
    q = st["x"][index]
    if gated:
        H = case["hidden"]
        q, s = q[:, :H].contiguous().view(FP8), q[:, H:].contiguous().view(torch.float32)
    else:
        s = st["x_scales"][index]
    x = (q.float().view(q.shape[0], -1, 128) * s[:, :, None]).view(q.shape)
    g = st["g_out"][index].float()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        at, xe, ge, w = index[a:b], x[a:b], g[a:b], st["w"][e].float()
        if gated:
            w2 = st["w2"][e].float()
            pre, up = xe @ w.t(), xe @ w2.t()
            act, slope = _act(pre, case["act"])
            d_pre, d_up = ge * up * slope, ge * act
            st["g_gate"][at], st["g_up"][at] = d_pre.to(BF16), d_up.to(BF16)
            st["g_x"][at] = (d_pre @ w + d_up @ w2).to(BF16)
            st["g_w"][e], st["g_w2"][e] = d_pre.t() @ xe, d_up.t() @ xe
        else:
            st["g_x"][at] = (ge @ w).to(BF16)
            st["g_w"][e] = ge.t() @ xe


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        _own(st)
    elif "mode" in case:
        _plain_product(st)
    else:
        _plain_move(st)
    if op == "sort" and case["form"] == "fp8":
        H = case["hidden"]
        return {"codes": st["out"][:, :H].view(FP8), "scales": st["out"][:, H:].view(torch.float32)}
    if op in ("sort", "sort_backward", "unsort"):
        return st["out"]
    if op == "unsort_backward":
        return {"y": st["g_y"], "w": st["g_w"]}
    if op == "linear_backward":
        return {"x": st["g_x"], "w": st["g_w"]}
    return {"x": st["g_x"], "gate": st["g_gate"], "up": st["g_up"], "w_gate": st["g_w"], "w_up": st["g_w2"]}


# ---------------------------------------------------------------------------
# Work, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, H = case["op"], case["hidden"]
    topk = _topk(case, 0)
    places = topk.size
    if "mode" not in case:
        rows = _places(case, topk)[2]
        if op == "sort":
            return {"bytes": (rows + places) * (H + H // 32 if case["form"] == "fp8" else 2 * H), "flops": 0}
        if op == "unsort_backward":
            return {"bytes": (rows + 2 * places) * 2 * H + 8 * places, "flops": 3 * places * H}
        weights = op == "unsort"
        return {"bytes": (rows + places) * 2 * H + 4 * places * weights, "flops": (1 + weights) * places * H}
    E, active = case["experts"], len(np.unique(topk))
    mats = 2 if op == "gated_backward" else 1
    K, N = (H, case["inter"]) if mats == 2 else (case["inter"], H)
    # gradients of every expert, weights of those that have rows; codes, scales, both rows' gradients, the gradient given
    moved = (E + active) * mats * N * K * 2 + places * (K + K // 32 + 2 * K + 2 * N + (4 * N if mats == 2 else 0))
    return {"bytes": moved, "flops": 2 * places * K * N * mats * (3 if mats == 2 else 2)}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_product(st) if "mode" in case else _exact_move(st)


def _exact_move(st):
    D = torch.float64
    case, row, entry = st["case"], st["row"], st["entry"]
    op, H = case["op"], case["hidden"]
    if op == "sort":
        x = st["x"].index_select(0, row)
        if case["form"] == "bf16":
            return x.to(D)
        return {"codes": x[:, :H].contiguous().view(FP8).to(D), "scales": x[:, H:].contiguous().view(torch.float32).to(D)}
    K = case["top_k"]
    if op == "unsort_backward":
        w = st["w"].to(D)[entry // K, entry % K]
        gy = torch.empty(st["g_y"].shape, dtype=D, device="cuda")
        dots = torch.empty(st["w"].shape, dtype=D, device="cuda")
        for a in range(0, len(row), 8192):
            g = st["g"].index_select(0, row[a:a + 8192]).to(D)
            gy[a:a + 8192] = torch.mul(w[a:a + 8192].unsqueeze(1), g)
            at = entry[a:a + 8192]
            dots[at // K, at % K] = torch.linalg.vecdot(g, st["y"][a:a + 8192].to(D))
        return {"y": gy, "w": dots}
    # the j-th entry of every row, for j = 0, 1, ...: no two of them share a row
    total = torch.zeros(st["out"].shape, dtype=D, device="cuda")
    order = torch.argsort(row, stable=True)
    per = torch.bincount(row, minlength=total.shape[0])
    first = torch.cumsum(per, 0) - per
    for j in range(int(per.max())):
        r = torch.nonzero(per > j).squeeze(1)
        at = order[first[r] + j]
        term = st["y"].index_select(0, at).to(D)
        if op == "unsort":
            term *= st["w"].to(D)[entry[at] // K, entry[at] % K].unsqueeze(1)
        total[r] += term
    return total


def _exact_product(st):
    D = torch.float64
    case, op = st["case"], st["case"]["op"]
    got = {}

    def like(name):
        return torch.zeros(st[name].shape, dtype=D, device="cuda")

    gated = op == "gated_backward"
    got["x"], got["w_gate" if gated else "w"] = like("g_x"), like("g_w")
    if gated:
        got["gate"], got["up"], got["w_up"] = like("g_gate"), like("g_up"), like("g_w2")
    for e in range(case["experts"]):
        at = st["index"][st["ends"][e]:st["ends"][e + 1]]
        if len(at) == 0:
            continue
        x, g, w = st["x"][at], st["g_out"][at].to(D), st["w"][e].to(D)
        if gated:
            H = case["hidden"]
            q, s = x[:, :H].contiguous().view(FP8), x[:, H:].contiguous().view(torch.float32)
        else:
            q, s = x, st["x_scales"][at]
        x = q.to(D) * torch.repeat_interleave(s.to(D), 128, dim=1)
        if not gated:
            got["x"][at], got["w"][e] = torch.mm(g, w), torch.mm(g.t(), x)
            continue
        w2 = st["w2"][e].to(D)
        p, u = torch.mm(x, w.t()), torch.mm(x, w2.t())
        if case["act"] == "silu":
            sig = torch.sigmoid(p)
            f, df = p * sig, sig + p * sig * (1 - sig)
        else:                                # 0.5 p (1 + tanh z) = p * sigmoid(2z)
            c = math.sqrt(8 / math.pi)
            sig = torch.sigmoid(c * (p + 0.044715 * p ** 3))
            f, df = p * sig, sig + p * sig * (1 - sig) * c * (1 + 0.134145 * p ** 2)
        dp, du = g * u * df, g * f
        got["gate"][at], got["up"][at] = dp, du
        got["x"][at] = torch.mm(dp, w) + torch.mm(du, w2)
        got["w_gate"][e], got["w_up"][e] = torch.mm(dp.t(), x), torch.mm(du.t(), x)
    return got
