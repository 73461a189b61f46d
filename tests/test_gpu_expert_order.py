"""Rows of ranks in expert order and back, with their adjoints, against references in 64 bits (bounds: order_util)."""
import numpy as np
import pytest
import torch

from gpu_util import A, I, dev, ep, get_map, host, need_gpu, say
from order_util import BF16, D, STALE, Ranks, near, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# sources, tokens, experts, entries, hidden, nodes, ranks a node
GEOMETRIES = [
    dict(S=1, T=1, E=4, K=1, H=16, nodes=1, per_node=1),        # one token, one entry, one rank
    dict(S=4, T=32, E=16, K=2, H=256, nodes=2, per_node=2),
    dict(S=3, T=37, E=24, K=3, H=1040, nodes=2, per_node=2),    # a row size that no tile divides
    dict(S=2, T=50, E=64, K=8, H=512, nodes=2, per_node=2),     # many entries share a row
    dict(S=1, T=70, E=64, K=9, H=272, nodes=4, per_node=4),     # more entries than a batch
    dict(S=1, T=33, E=32, K=32, H=128, nodes=1, per_node=2),    # every expert
    dict(S=1, T=130, E=256, K=8, H=7168, nodes=8, per_node=8),
    dict(S=1, T=20, E=1024, K=17, H=4112, nodes=16, per_node=64),
    dict(S=1, T=9, E=8, K=8, H=16384, nodes=1, per_node=1),     # one rank: a token's entries are one row
]
ids = [f"{g['S']}x{g['T']}-{g['E']}-{g['K']}-{g['H']}" for g in GEOMETRIES]


def invalid(topk, E, seed):
    """A routing with entries out of range, repeated ones, and a token without any valid one."""
    rng = np.random.default_rng(seed)
    t = topk.copy()
    t[rng.random(t.shape) < 0.1] = -1
    t[rng.random(t.shape) < 0.05] = E
    if t.shape[1] > 1:
        again = rng.random(t.shape[0]) < 0.3
        t[again, 1] = t[again, 0]
    t[t.shape[0] // 2] = -5
    return t


@pytest.mark.parametrize("spoilt", [False, True], ids=["valid", "invalid"])
@pytest.mark.parametrize("g", GEOMETRIES, ids=ids)
def test_places_and_counts(g, spoilt):
    say(f"places {g} invalid={spoilt}")
    topk = np.argsort(np.random.default_rng(2).random((g["S"] * g["T"], g["E"])), axis=1)[:, :g["K"]].astype(np.int32)
    with Ranks(**g, topk=invalid(topk, g["E"], 3) if spoilt else topk) as r:
        np.testing.assert_array_equal(get_map(r.handle, A.EP_MAP_HT_SORTED_ROW), r.place)
        np.testing.assert_array_equal(get_map(r.handle, A.EP_MAP_HT_SORTED_COUNT), r.count)
        np.testing.assert_array_equal(get_map(r.handle, A.EP_MAP_HT_EXPERT_COUNT), r.rank_count)
        # the ranks' map holds each row once
        first = np.array([[k == list(x).index(x[k]) for k in range(r.K)] for x in r.row]) & (r.row >= 0)
        np.testing.assert_array_equal(get_map(r.handle, A.EP_MAP_HT_ROW), np.where(first, r.row, -1))
        # the places are the rows that the per-expert stage 2 gives
        cfg = dict(r.group.config, ht_stage2="expert")
        other = ep.ep_create_group(**cfg)
        h = ep.ep_create_handle(other, r.idx)
        np.testing.assert_array_equal(get_map(h, A.EP_MAP_HT_ROW), r.place)
        ep.ep_destroy_group(other)
        assert (ep.ep_get_device_error(r.group) != 0) == spoilt


def test_places_of_a_routed_handle():
    """ep_route_handle (routing and counting in one kernel) gives the same places as a handle of its entries."""
    say("places of a routed handle")
    w = I.HT_PREFILL.with_(num_src_ranks=2, tokens_per_rank=150, hidden=128, seed=9)
    with Ranks(S=2, T=150, E=256, K=8, H=128, nodes=8, per_node=8, payload="fp8", max_nodes_per_token=4) as r:
        topk = torch.empty((300, 8), dtype=torch.int32, device="cuda")
        h = ep.ep_route_handle(r.group, dev(I.scores_for(w)), topk)
        with Ranks(S=2, T=150, E=256, K=8, H=128, nodes=8, per_node=8, topk=host(topk)) as q:
            for m in (A.EP_MAP_HT_SORTED_ROW, A.EP_MAP_HT_SORTED_COUNT, A.EP_MAP_HT_ROW, A.EP_MAP_HT_EXPERT_COUNT):
                np.testing.assert_array_equal(get_map(h, m), get_map(q.handle, m))
            np.testing.assert_array_equal(get_map(h, A.EP_MAP_HT_SORTED_ROW), q.place)


def check_sort(r, x, out):
    assert torch.equal(out[:r.places].view(torch.uint8), x[r.row_of].view(torch.uint8))
    assert bool((out[r.places:] == STALE).all())


def check_all(r, pad=0):
    """All four calls with rows behind those in use, which stay as they were."""
    x, out = r.at_rows(1, 3, pad), r.stale(r.places + 2, pad)
    ep.ep_expert_sort(r.handle, x, out)
    check_sort(r, x, out)
    y, w = r.at_places(2, 2, pad), r.weights(3)
    rows = r.stale(r.rows + 3, pad)
    ep.ep_expert_unsort(r.handle, y, w, rows)
    near(rows[:r.rows], *r.unsorted(y, w), "unsort")
    assert bool((rows[r.rows:] == STALE).all())
    rows = r.stale(r.rows + 3, pad)
    ep.ep_expert_sort_backward(r.handle, y, rows)
    near(rows[:r.rows], *r.unsorted(y, None), "sort, backward")
    assert bool((rows[r.rows:] == STALE).all())
    dy, dw = r.stale(r.places + 2, pad), torch.full((r.n, r.K), STALE, device="cuda")
    ep.ep_expert_unsort_backward(r.handle, x, w, dy, expert_out=y, grad_weights=dw)
    near(dy[:r.places], *r.spread(x, w), "unsort, backward")
    near(dw, *r.dots(x, y), "weights")
    assert bool((dy[r.places:] == STALE).all())
    alone = r.stale(r.places + 2, pad)
    ep.ep_expert_unsort_backward(r.handle, x, w, alone)
    assert torch.equal(alone, dy)


@pytest.mark.parametrize("g", GEOMETRIES, ids=ids)
def test_moves(g):
    say(f"moves {g}")
    with Ranks(**g, seed=4) as r:
        check_all(r)
        check_all(r, pad=24)
        assert ep.ep_get_device_error(r.group) == 0


@pytest.mark.parametrize("g", GEOMETRIES[1:], ids=ids[1:])
def test_moves_with_invalid_entries(g):
    say(f"moves {g}, invalid entries")
    topk = np.argsort(np.random.default_rng(5).random((g["S"] * g["T"], g["E"])), axis=1)[:, :g["K"]].astype(np.int32)
    with Ranks(**g, topk=invalid(topk, g["E"], 6)) as r:
        check_all(r)


@pytest.mark.parametrize("H", [128, 384, 512, 7168])
def test_packed_rows(H):
    """The dispatch's FP8 rows: codes and scales byte for byte, from its buffer; what lies behind a row's bytes."""
    say(f"packed rows, hidden {H}")
    used = H + H // 32
    pitch = -(-used // 128) * 128
    with Ranks(S=2, T=45, E=32, K=5, H=H, nodes=2, per_node=4, payload="fp8") as r:
        ep.ep_dispatch(r.handle, normal((r.n, H), 7, 3.0))
        rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_HT_STAGE2)
        want = rows[:r.rows][r.row_of]
        for width, stride in ((used, pitch), (pitch, pitch), (used, used + 16 - used % 16 + 64), (pitch + 16, pitch + 32)):
            whole = torch.full((r.places + 2, stride), 77, dtype=torch.uint8, device="cuda")
            out = whole[:, :width]
            ep.ep_expert_sort(r.handle, rows, out)
            assert torch.equal(whole[:r.places, :used], want)
            filled = pitch if width >= pitch else used
            assert not bool(whole[:r.places, used:filled].any())
            assert bool((whole[:r.places, filled:] == 77).all()) and bool((whole[r.places:] == 77).all())
        # BF16 rows of an FP8 group
        x, out = r.at_rows(8), r.stale(r.places)
        ep.ep_expert_sort(r.handle, x, out)
        check_sort(r, x, out)


def test_packed_bf16_rows():
    say("packed BF16 rows")
    with Ranks(S=1, T=60, E=16, K=4, H=272, payload="bf16") as r:
        ep.ep_dispatch(r.handle, normal((r.n, 272), 7))
        rows = ep.ep_handle_get_buffer(r.handle, A.EP_BUF_HT_STAGE2)
        out = torch.zeros((r.places, 640), dtype=torch.uint8, device="cuda")[:, :544]
        ep.ep_expert_sort(r.handle, rows, out)
        assert torch.equal(out, rows[:r.rows][r.row_of])


@pytest.mark.parametrize("K", [4, 12])
def test_tensors_that_are_too_short(K):
    """What the tensors do not hold is left out, the others' sums are whole, and the error word says so."""
    say(f"short tensors, {K} entries")
    with Ranks(S=1, T=90, E=32, K=K, H=256) as r:
        x, y, w = r.at_rows(1), r.at_places(2), r.weights(3)
        cut, held = r.places * 2 // 3, r.rows // 2
        out = r.stale(r.places)
        ep.ep_expert_sort(r.handle, x[:held], out[:cut])
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        on = (torch.arange(r.places, device="cuda") < cut) & (r.row_of < held)
        assert torch.equal(out[on], x[r.row_of[on]]) and bool((out[~on] == STALE).all())
        rows = r.stale(r.rows)
        ep.ep_expert_unsort(r.handle, y[:cut], w, rows[:held])
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        some = y.clone()
        some[cut:] = 0
        v, b = r.unsorted(some, w)
        near(rows[:held], v[:held], b[:held])
        assert bool((rows[held:] == STALE).all())
        dy, dw = r.stale(r.places), torch.full((r.n, r.K), STALE, device="cuda")
        ep.ep_expert_unsort_backward(r.handle, x[:held], w, dy[:cut], expert_out=y, grad_weights=dw)
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        v, b = r.spread(x, w)
        near(dy[on], v[on], b[on])
        assert bool((dy[~on] == STALE).all())
        v, b = r.dots(x, y)
        gone = torch.ones(r.n * r.K, dtype=torch.bool, device="cuda")
        gone[r.entry[on]] = False
        near(dw, v.masked_fill(gone.view(r.n, r.K), 0), b)
        none = torch.empty((0, 256), dtype=BF16, device="cuda")
        for call in (lambda: ep.ep_expert_sort(r.handle, none, none),
                     lambda: ep.ep_expert_unsort(r.handle, none, w, none),
                     lambda: ep.ep_expert_sort_backward(r.handle, none, none),
                     lambda: ep.ep_expert_unsort_backward(r.handle, none, w, none, expert_out=none, grad_weights=dw)):
            call()
            assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        assert bool((dw == 0).all())


def test_no_tokens():
    say("no tokens")
    with Ranks(S=2, T=0, E=8, K=2, H=64, topk=np.zeros((0, 2), np.int32)) as r:
        x, w = r.stale(3), torch.empty((0, 2), device="cuda")
        out = x.clone()
        ep.ep_expert_sort(r.handle, x, out)
        ep.ep_expert_unsort(r.handle, x, w, out)
        ep.ep_expert_sort_backward(r.handle, x, out)
        ep.ep_expert_unsort_backward(r.handle, x, w, out, expert_out=x, grad_weights=w)
        assert bool((out == STALE).all())
        assert not get_map(r.handle, A.EP_MAP_HT_SORTED_COUNT).any()
        dw = torch.full((8, 32, 64), 9.0, device="cuda")
        ep.ep_expert_linear_backward(r.handle, x, torch.zeros((8, 32, 64), dtype=BF16, device="cuda"),
                                     torch.zeros((3, 32), dtype=BF16, device="cuda"), grad_w=dw)
        assert not bool(dw.any())


def test_values_that_are_not_finite_stay_in_their_rows():
    """Infinities and NaN of one place reach its rank's row alone, its token's other rows nothing; a zero weight of an
    infinite row gives NaN as the formula does."""
    say("infinity and NaN")
    with Ranks(S=1, T=60, E=16, K=4, H=256) as r:
        y, w = r.at_places(1), r.weights(2)
        clean = r.stale(r.rows)
        ep.ep_expert_unsort(r.handle, y, w, clean)
        y[7, 3], y[20, 250] = float("inf"), float("nan")
        w.view(-1)[r.entry[7]] = 0
        want, _ = r.unsorted(y, w)
        got = r.stale(r.rows)
        ep.ep_expert_unsort(r.handle, y, w, got)
        assert torch.equal(got.isfinite(), want.isfinite())
        assert bool(got[r.row_of[7], 3].isnan()) and bool(got[r.row_of[20], 250].isnan())
        same = torch.ones(r.rows, dtype=torch.bool, device="cuda")
        same[r.row_of[[7, 20]]] = False
        assert torch.equal(got[same], clean[same])
        # the largest values round as bf16 does, to infinity past the largest finite one
        big = torch.full_like(y, torch.finfo(BF16).max)
        ones = torch.ones_like(w)
        ep.ep_expert_sort_backward(r.handle, big, got)
        per = torch.bincount(r.row_of, minlength=r.rows)
        assert torch.equal(got[:, 0].isinf(), per > 1) and bool((got[per == 1] == torch.finfo(BF16).max).all())
        dy = r.stale(r.places)
        ep.ep_expert_unsort_backward(r.handle, big[:r.rows], ones, dy)
        assert bool((dy == torch.finfo(BF16).max).all())


def test_far_rows():
    """Rows more than 2^31 bytes and 2^31 elements apart from the first."""
    say("far rows")
    far = 40 * 1024 * 1024 + 8
    with Ranks(S=1, T=30, E=8, K=3, H=64) as r:
        def spread_out(rows, src):
            t = torch.empty((rows * far,), dtype=BF16, device="cuda").as_strided((rows, 64), (far, 1))
            t.copy_(src[:rows])
            return t
        assert r.places * far > 2 ** 31
        x = spread_out(r.rows, r.at_rows(1))
        y = spread_out(r.places, r.stale(r.places))
        ep.ep_expert_sort(r.handle, x, y)
        check_sort(r, x.contiguous(), y.contiguous())
        w = r.weights(2)
        ep.ep_expert_unsort(r.handle, y, w, x)
        near(x, *r.unsorted(y, w))
        dw = torch.empty_like(w)
        dy = spread_out(r.places, r.stale(r.places))
        ep.ep_expert_unsort_backward(r.handle, x, w, dy, expert_out=y, grad_weights=dw)
        near(dy, *r.spread(x, w))
        near(dw, *r.dots(x, y))


def test_many_tokens():
    """More tokens than a launch's second dimension holds."""
    say("many tokens")
    T = 70001
    topk = np.zeros((T, 1), np.int32)
    topk[:, 0] = np.random.default_rng(1).integers(0, 4, T)
    with Ranks(S=1, T=T, E=4, K=1, H=16, topk=topk) as r:
        check_all(r)


def test_the_combine_behind_and_its_adjoint():
    """unsort, then the combine of the ranks' rows; ep_combine_backward gives every rank's row its token's gradient."""
    say("combine behind the way back")
    with Ranks(S=2, T=60, E=32, K=6, H=512, nodes=2, per_node=4) as r:
        g = normal((r.n, r.H), 1)
        rows = r.stale(r.rows + 1)
        ep.ep_combine_backward(r.handle, g, None, rows)
        token = torch.zeros(r.rows, dtype=torch.int64, device="cuda")
        token[r.row_of] = r.entry // r.K
        assert torch.equal(rows[:r.rows], g[token]) and bool((rows[r.rows:] == STALE).all())
        y, w = r.at_places(2), r.weights(3)
        ep.ep_expert_unsort(r.handle, y, w, rows)
        out = torch.empty((r.n, r.H), dtype=BF16, device="cuda")
        ep.ep_combine(r.handle, rows, None, out)
        want = torch.zeros((r.n, r.H), dtype=D, device="cuda").index_add_(0, token, rows[:r.rows].to(D))
        mag = torch.zeros((r.n, r.H), dtype=D, device="cuda").index_add_(0, token, rows[:r.rows].to(D).abs())
        near(out, want, r.K * 2.0 ** -24 * mag + 2.0 ** -8 * 1.01 * want.abs())
        for kw in (dict(topk_weights=w), dict(topk_weights=None, expert_out=rows),
                   dict(topk_weights=None, expert_out=rows, grad_weights=w)):
            with pytest.raises(ep.EpError) as ei:
                ep.ep_combine_backward(r.handle, g, grad_expert_out=rows, **kw)
            assert ei.value.status == A.EP_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("spoilt", [False, True], ids=["valid", "invalid"])
@pytest.mark.parametrize("g", GEOMETRIES[1:], ids=ids[1:])
def test_the_combine_adjoint(g, spoilt):
    """Every rank's row of a token is a copy of the token's gradient: strided, in tensors that hold fewer rows, with a cap
    on the CUs, captured."""
    say(f"combine adjoint {g}, {'invalid' if spoilt else 'valid'} entries")
    topk = np.argsort(np.random.default_rng(7).random((g["S"] * g["T"], g["E"])), axis=1)[:, :g["K"]].astype(np.int32)
    with Ranks(**g, topk=invalid(topk, g["E"], 8) if spoilt else topk) as r:
        ep.ep_get_device_error(r.group)   # of the entries
        token = torch.zeros(r.rows, dtype=torch.int64, device="cuda")
        token[r.row_of] = r.entry // r.K
        grad = normal((r.n, r.H + 8), 1)[:, :r.H]
        want = grad[token]

        def rows(more, pad=0):
            return torch.full((r.rows + more, r.H + pad), STALE, dtype=BF16, device="cuda")

        wide = rows(2, 16)
        ep.ep_combine_backward(r.handle, grad, None, wide[:, :r.H])
        assert torch.equal(wide[:r.rows, :r.H], want)
        assert bool((wide[r.rows:] == STALE).all()) and bool((wide[:, r.H:] == STALE).all())
        assert ep.ep_get_device_error(r.group) == 0
        short = rows(0)
        keep = r.rows // 2
        ep.ep_combine_backward(r.handle, grad, None, short[:keep])
        assert torch.equal(short[:keep], want[:keep]) and bool((short[keep:] == STALE).all())
        assert ep.ep_get_device_error(r.group) == A.EP_DEVERR_ROW_RANGE
        capped = ep.ep_create_group(**dict(r.group.config, num_cus=1))
        h = ep.ep_create_handle(capped, r.idx)
        few = rows(0)
        ep.ep_combine_backward(h, grad, None, few)
        assert torch.equal(few, want)
        ep.ep_destroy_group(capped)
        out, graph = rows(0), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ep.ep_combine_backward(r.handle, grad, None, out)
        for turn in range(3):
            grad.copy_(normal((r.n, r.H), 20 + turn))
            out.fill_(STALE)
            graph.replay()
            assert torch.equal(out, grad[token]), turn


def refused(status, fn, *args, **kw):
    with pytest.raises(ep.EpError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status, (fn.__name__, ei.value)


def test_refusals():
    say("refusals")
    bad = A.EP_ERR_INVALID_ARGUMENT
    with Ranks(S=1, T=20, E=8, K=2, H=256, payload="fp8") as r:
        x, y, w = r.at_rows(1), r.at_places(2), r.weights(3)
        out, rows, dw = r.stale(r.places), r.stale(r.rows), torch.full((r.n, r.K), STALE, device="cuda")
        u8 = torch.zeros((r.places, 384), dtype=torch.uint8, device="cuda")
        wrong_rows = [x.float(), x[:, :128], x.t(), x.view(-1), x.view(r.rows, 16, 16), torch.empty_like(x).half(),
                      torch.empty(r.rows * 256 + 4, dtype=BF16, device="cuda")[4:].view(r.rows, 256),
                      torch.empty((r.rows, 260), dtype=BF16, device="cuda")[:, :256]]
        for t in wrong_rows:
            refused(bad, ep.ep_expert_sort, r.handle, t, out)
            refused(bad, ep.ep_expert_sort, r.handle, x, t)
            refused(bad, ep.ep_expert_sort_backward, r.handle, t, rows)
            refused(bad, ep.ep_expert_sort_backward, r.handle, y, t)
            refused(bad, ep.ep_expert_unsort, r.handle, t, w, rows)
            refused(bad, ep.ep_expert_unsort, r.handle, y, w, t)
            refused(bad, ep.ep_expert_unsort_backward, r.handle, t, w, out)
            refused(bad, ep.ep_expert_unsort_backward, r.handle, x, w, t)
            refused(bad, ep.ep_expert_unsort_backward, r.handle, x, w, out, expert_out=t)
        refused(bad, ep.ep_expert_sort, r.handle, u8, out)                 # packed to BF16
        refused(bad, ep.ep_expert_sort, r.handle, x, u8)
        refused(bad, ep.ep_expert_sort, r.handle, u8[:, :256], u8)         # narrower than a row's 264 bytes
        refused(bad, ep.ep_expert_sort, r.handle, u8, u8[:, :256])
        wide = torch.zeros((r.places, 392), dtype=torch.uint8, device="cuda")
        refused(bad, ep.ep_expert_sort, r.handle, wide, u8)                # rows off 16 bytes
        for t in (w.double(), w[:-1], w.t(), w.bfloat16(), torch.empty((r.n, 4), device="cuda")[:, :2], w.view(-1)):
            if t.dtype == torch.float64:
                continue                                                   # no such type in a descriptor
            refused(bad, ep.ep_expert_unsort, r.handle, y, t, rows)
            refused(bad, ep.ep_expert_unsort_backward, r.handle, x, t, out)
            refused(bad, ep.ep_expert_unsort_backward, r.handle, x, w, out, expert_out=y, grad_weights=t)
        refused(bad, ep.ep_expert_unsort, r.handle, y, None, rows)
        refused(bad, ep.ep_expert_unsort_backward, r.handle, x, None, out)
        refused(bad, ep.ep_expert_unsort_backward, r.handle, x, w, out, grad_weights=dw)
        for stage2, mode in (("expert", "ht"), ("rank", "ht"), ("rank_sorted", "ll")):
            g = ep.ep_create_group(**dict(r.group.config, ht_stage2=stage2, mode=mode))
            h = ep.ep_create_handle(g, r.idx)
            refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_sort, h, x, out)
            refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_sort_backward, h, y, rows)
            refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_unsort, h, y, w, rows)
            refused(A.EP_ERR_UNSUPPORTED, ep.ep_expert_unsort_backward, h, x, w, out)
            for m in (A.EP_MAP_HT_SORTED_ROW, A.EP_MAP_HT_SORTED_COUNT):
                refused(bad, ep.ep_handle_get_map, h, m)
            ep.ep_destroy_group(g)
        torch.cuda.synchronize()
        for t in (out, rows, dw):
            assert bool((t == STALE).all()), "a refused call wrote"
        assert ep.ep_get_device_error(r.group) == 0
        gone = ep.ep_create_handle(r.group, r.idx)
        ep.ep_destroy_handle(gone)
        refused(bad, ep.ep_expert_sort, gone, x, out)
        with pytest.raises(ValueError):
            ep.ep_expert_sort(r.handle, x.cpu(), out)


def test_streams_and_repeats():
    """The same bits again; calls of one handle on several streams at once, behind each stream's own work; a cap on
    the CUs; a second handle of the group."""
    say("streams and repeats")
    with Ranks(S=2, T=300, E=64, K=6, H=1024, nodes=2, per_node=4, max_handles=2) as r:
        other = ep.ep_create_handle(r.group, r.idx.flip(0).contiguous())
        x, y, w = r.at_rows(1), r.at_places(2), r.weights(3)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(1_000_000)
                late_x, late_y, late_w = x.clone(), y.clone(), w.clone()
                out, rows, back, dy, dw = (torch.empty_like(late_y), torch.empty_like(late_x), torch.empty_like(late_x),
                                           torch.empty_like(late_y), torch.empty_like(late_w))
                ep.ep_expert_sort(other, late_x, torch.empty_like(late_y))
                ep.ep_expert_sort(r.handle, late_x, out)
                ep.ep_expert_unsort(r.handle, late_y, late_w, rows)
                ep.ep_expert_sort_backward(r.handle, late_y, back)
                ep.ep_expert_unsort_backward(r.handle, late_x, late_w, dy, expert_out=late_y, grad_weights=dw)
                got.append([out, rows, back, dy, dw, late_x, late_y, late_w])
        torch.cuda.synchronize()
        check_sort(r, x, got[0][0])
        near(got[0][1], *r.unsorted(y, w))
        near(got[0][2], *r.unsorted(y, None))
        near(got[0][3], *r.spread(x, w))
        near(got[0][4], *r.dots(x, y))
        for g in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(got[0], g))
        capped = ep.ep_create_group(**dict(r.group.config, num_cus=3))
        h = ep.ep_create_handle(capped, r.idx)
        again = [torch.empty_like(t) for t in got[0][:5]]
        ep.ep_expert_sort(h, x, again[0])
        ep.ep_expert_unsort(h, y, w, again[1])
        ep.ep_expert_sort_backward(h, y, again[2])
        ep.ep_expert_unsort_backward(h, x, w, again[3], expert_out=y, grad_weights=again[4])
        assert all(torch.equal(a, b) for a, b in zip(got[0], again))
        ep.ep_destroy_group(capped)


def test_captured():
    """A handle made and its rows moved inside a graph, replayed with new entries and rows, with eager calls between."""
    say("captured moves")
    with Ranks(S=1, T=80, E=32, K=4, H=512, nodes=2, per_node=4, max_handles=2) as r:
        idx, w = r.idx.clone(), r.weights(1)
        x, y = torch.zeros((r.n * r.K, r.H), dtype=BF16, device="cuda"), torch.zeros((r.n * r.K, r.H), dtype=BF16, device="cuda")
        outs = [torch.zeros_like(x) for _ in range(4)] + [torch.zeros_like(w)]

        def step(h, o):
            ep.ep_expert_sort(h, x, o[0])
            ep.ep_expert_unsort(h, y, w, o[1])
            ep.ep_expert_sort_backward(h, y, o[2])
            ep.ep_expert_unsort_backward(h, x, w, o[3], expert_out=y, grad_weights=o[4])

        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            h = ep.ep_create_handle(r.group, idx)
            step(h, outs)
        for turn in range(4):
            with Ranks(S=1, T=80, E=32, K=4, H=512, nodes=2, per_node=4, seed=10 + turn) as q:
                idx.copy_(q.idx)
                x[:q.rows], y[:q.places] = q.at_rows(20 + turn), q.at_places(30 + turn)
                w.copy_(q.weights(40 + turn))
                for o in outs:
                    o.fill_(STALE)
                graph.replay()
                eager = [torch.full_like(o, STALE) for o in outs]
                step(q.handle, eager)
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(outs, eager)), turn
                near(outs[1][:q.rows], *q.unsorted(y, w))
                near(outs[4], *q.dots(x, y))
