"""The stage-2 kind with expert order on the host: which configurations take it, what it costs in memory, and what its
calls refuse without a handle (CPU only; groups on host memory)."""
import ctypes

import pytest
import torch

from combine_ep_route_amd import _abi as A, ep
from test_abi_host import FAKE, HostPool, _cfg, _create, _t

BAD = A.EP_ERR_INVALID_ARGUMENT
KINDS = (A.EP_HT_STAGE2_PER_RANK, A.EP_HT_STAGE2_PER_RANK_SORTED)


def test_memory_of_the_places():
    """Per handle three maps of n*K, counts per expert and per tile; with max_handles = 3 that three times."""
    sizes = {}
    for kind in KINDS:
        pool = HostPool()
        st, g = _create(_cfg(pool, ht_stage2=kind, max_tokens_per_rank=256, max_handles=3))
        assert st == A.EP_OK
        b = ctypes.c_int64()
        assert A.lib().ep_group_memory(g, ctypes.byref(b)) == A.EP_OK
        sizes[kind] = b.value
        view = A.EpTensor()
        assert A.lib().ep_get_buffer(g, A.EP_BUF_HT_STAGE2_TOPK, ctypes.byref(view)) == A.EP_OK
        assert A.lib().ep_destroy_group(g) == A.EP_OK
    cfg = _cfg(None)
    n, K, E = 256 * cfg.num_src_ranks, cfg.top_k, cfg.num_experts
    extra = 3 * n * K * 4 + E * 4 + n // 16 * E * 4
    grown = sizes[KINDS[1]] - sizes[KINDS[0]]
    assert 3 * extra <= grown <= 3 * (extra + 6 * 256)


@pytest.mark.parametrize("mode", [A.EP_MODE_HT, A.EP_MODE_LL])
def test_accepted_in_both_modes(mode):
    """LL ignores the stage-2 kind, this one too."""
    pool = HostPool()
    st, g = _create(_cfg(pool, mode=mode, ht_stage2=A.EP_HT_STAGE2_PER_RANK_SORTED, max_tokens_per_rank=16))
    assert st == A.EP_OK
    assert A.lib().ep_destroy_group(g) == A.EP_OK


@pytest.mark.parametrize("kind", [2, 4, 5, 7, -3])
def test_other_kinds_are_refused(kind):
    pool = HostPool()
    st, _ = _create(_cfg(pool, ht_stage2=kind))
    assert st == BAD and pool.calls == 0


def test_calls_without_a_handle():
    t = _t(FAKE, A.EP_DTYPE_BF16, [4, 256])
    w = _t(FAKE, A.EP_DTYPE_F32, [4, 2])
    r = ctypes.byref
    lib = A.lib()
    group = ctypes.create_string_buffer(4096)   # memory that is no handle
    for h in (None, ctypes.addressof(group)):
        assert lib.ep_expert_sort(h, r(t), r(t), None) == BAD
        assert lib.ep_expert_sort_backward(h, r(t), r(t), None) == BAD
        assert lib.ep_expert_unsort(h, r(t), r(w), r(t), None) == BAD
        assert lib.ep_expert_unsort_backward(h, r(t), None, r(w), r(t), None, None) == BAD


def test_places_without_a_handle_are_refused():
    """The layout without a group has no places: asking for them is an error, not a tensor left as it was."""
    topk = torch.zeros((4, 2), dtype=torch.int32)
    for which in (A.EP_MAP_HT_SORTED_ROW, A.EP_MAP_HT_SORTED_COUNT):
        with pytest.raises(ValueError):
            ep.ep_layout_noalloc(topk, {which: torch.zeros((4, 2), dtype=torch.int32)}, mode="ht",
                                 ht_stage2="rank_sorted", top_k=2)
