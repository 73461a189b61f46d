"""Device memory of an LL handle slot: the experts' row list is part of it only where the products read one (CPU only;
groups on host memory that is never read)."""
import ctypes

import pytest

from combine_ep_route_amd import _abi as A
from test_abi_host import HostPool, _cfg, _create


def slot_bytes(**kw):
    """What one more handle slot adds to a group."""
    got = []
    for handles in (1, 2):
        pool = HostPool()
        st, g = _create(_cfg(pool, mode=A.EP_MODE_LL, max_handles=handles, **kw))
        assert st == A.EP_OK
        b = ctypes.c_int64()
        assert A.lib().ep_group_memory(g, ctypes.byref(b)) == A.EP_OK
        got.append(b.value)
        A.lib().ep_destroy_group(g)
    return got[1] - got[0]


def up(values):
    return (values * 4 + 255) // 256 * 256


@pytest.mark.parametrize("sources,experts,listed", [(1, 256, False), (2, 64, False), (8, 16, False), (4, 32, False),
                                                    (2, 72, True), (8, 24, True), (9, 16, True), (64, 64, True)])
def test_row_list_only_where_it_is_read(sources, experts, listed):
    T, K = 100, 2
    nodes, ranks = 8, experts // 8
    n, tiles = sources * T, sources * ((T + 15) // 16)
    want = 3 * up(n * K) + up(n * nodes) + up(experts * sources) + up(tiles * experts) + up(tiles * nodes)
    if listed:
        want += up(experts) + up(n * K)
    got = slot_bytes(num_nodes=nodes, ranks_per_node=ranks, num_experts=experts, num_src_ranks=sources, top_k=K,
                     max_nodes_per_token=0, max_tokens_per_rank=T, hidden=128)
    assert got == want
