"""Calls of more rows than a single launch holds (a grid dimension counts its threads in 32 bits).  Rows are compared
with the same rows of small calls, bit for bit.  Tensors are left as allocated outside the rows that are compared."""
import pytest
import torch

from expert_util import BF16, normal
from gpu_util import ep, need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def room(gib):
    free = torch.cuda.mem_get_info()[0] >> 30
    if free < gib + 4:
        pytest.skip(f"{gib} GiB of device memory, {free} free")


def one_expert(H, payload="bf16"):
    return ep.ep_create_group(mode="ht", num_nodes=1, ranks_per_node=1, num_experts=1, top_k=1, max_nodes_per_token=0,
                              hidden=H, max_tokens_per_rank=1, num_src_ranks=1, payload=payload)


@pytest.mark.parametrize("gate", ["none", "token"])
def test_norm_of_the_most_rows(gate):
    """2^22 rows of 1024 threads each: 2^32 threads."""
    n, H = 1 << 22, 7696
    say(f"residual norm of {n} rows, gate {gate}")
    room(185 if gate == "token" else 124)
    g = one_expert(H)
    w = 1 + normal((H,), 1, 0.2, torch.float32)
    x, y = (torch.empty((n, H), dtype=BF16, device="cuda") for _ in range(2))
    t = torch.empty((n, H), dtype=BF16, device="cuda") if gate == "token" else None
    kw = dict(w_post=w, residual_scale=0.5, block_scale=2.0)
    parts, want = [slice(0, 300), slice(n // 2 - 150, n // 2 + 150), slice(n - 300, n)], []
    for i, at in enumerate(parts):
        small = [normal((300, H), 10 * i + k) for k in range(3)]
        x[at], y[at] = small[0], small[1]
        if t is not None:
            t[at] = small[2]
        res, out = torch.empty((300, H), dtype=BF16, device="cuda"), torch.empty((300, H), dtype=BF16, device="cuda")
        ep.ep_residual_norm(g, small[1], small[0], res, out, w, gate=small[2] if t is not None else None, **kw)
        want.append((res, out))
    ep.ep_residual_norm(g, y, x, x, y, w, gate=t, **kw)      # in place
    torch.cuda.synchronize()
    for at, (res, out) in zip(parts, want):
        assert torch.equal(x[at], res) and torch.equal(y[at], out), at
    ep.ep_destroy_group(g)


def test_quantize_and_dequantize_more_rows_than_a_grid_holds():
    """Over 2^26 rows of 128 values: ep_quantize gives every row a wave, ep_dequantize_rows a workgroup of one."""
    H, part, parts, rest = 128, 1 << 20, 64, 5
    n = parts * part + rest
    say(f"quantise and dequantise {n} rows")
    room(60)
    g = one_expert(H, "fp8")
    base = normal((part, H), 3, 4.0)
    q0, s0 = torch.empty((part, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((part, 1), device="cuda")
    ep.ep_quantize(g, base, q0, s0)
    x = torch.empty((n, H), dtype=BF16, device="cuda")
    x[:parts * part].view(parts, part, H).copy_(base)
    x[parts * part:] = base[:rest]
    q, s = torch.empty((n, H), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((n, 1), device="cuda")
    ep.ep_quantize(g, x, q, s)
    torch.cuda.synchronize()
    codes = q.view(torch.uint8)
    for i in range(parts + 1):
        at = slice(i * part, min(n, (i + 1) * part))
        m = at.stop - at.start
        assert torch.equal(codes[at], q0[:m].view(torch.uint8)) and torch.equal(s[at], s0[:m]), i

    rows = torch.zeros((n, H + 16), dtype=torch.uint8, device="cuda")   # codes, one scale, padding
    rows[:, :H] = codes
    rows[:, H:H + 4] = s.view(torch.uint8)
    y0 = torch.empty((part, H), dtype=BF16, device="cuda")
    ep.ep_dequantize_rows(g, rows[:part], y0)
    del x, q, s, codes
    y = torch.empty((n, H), dtype=BF16, device="cuda")
    ep.ep_dequantize_rows(g, rows, y)
    torch.cuda.synchronize()
    for i in range(parts + 1):
        at = slice(i * part, min(n, (i + 1) * part))
        assert torch.equal(y[at], y0[:at.stop - at.start]), i
    ep.ep_destroy_group(g)
