"""What ep_residual_norm and its backward pass refuse before any HIP call, and the experts' products without
a handle (CPU only; groups on host memory, addresses that are never read)."""
import ctypes

import pytest

from combine_ep_route_amd import _abi as A
from test_abi_host import FAKE, HostPool, _cfg, _create, _t

N, H = 5, 256
BAD = A.EP_ERR_INVALID_ARGUMENT


@pytest.fixture
def group():
    pool = HostPool()
    st, g = _create(_cfg(pool, hidden=H))
    assert st == A.EP_OK
    yield g
    A.lib().ep_destroy_group(g)


def _rows(**kw):
    d = dict(data=FAKE, dtype=A.EP_DTYPE_BF16, sizes=[N, H])
    d.update(kw)
    return _t(d["data"], d["dtype"], d["sizes"], d.get("strides"), d.get("tag", A.EP_TAG_NONE))


def _vec(n=H, dtype=A.EP_DTYPE_F32, data=FAKE):
    return _t(data, dtype, [n])


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _forward(group, a=1.0, b=1.0, eps=1e-6, **over):
    t = dict(y=_rows(), x=_rows(), w_post=_vec(), gate=None, w_pre=_vec(), out_x=_rows(), out_n=_rows())
    t.update(over)
    return A.lib().ep_residual_norm(group, _ref(t["y"]), _ref(t["x"]), _ref(t["w_post"]), _ref(t["gate"]),
                                    _ref(t["w_pre"]), a, b, eps, _ref(t["out_x"]), _ref(t["out_n"]), None)


WRONG_ROWS = [dict(dtype=A.EP_DTYPE_F16), dict(sizes=[N + 1, H]), dict(sizes=[N, H - 16]), dict(data=FAKE + 8),
              dict(strides=[H + 4, 1]), dict(strides=[H, 2]), dict(strides=[H - 16, 1]), dict(data=None),
              dict(sizes=[N * H]), dict(tag=A.EP_TAG_SCALES)]
WRONG_VECTORS = [_vec(H - 16), _vec(dtype=A.EP_DTYPE_F16), _vec(data=FAKE + 4), _vec(data=None),
                 _t(FAKE, A.EP_DTYPE_F32, [2, H]), _t(FAKE, A.EP_DTYPE_F32, [H], [2])]


@pytest.mark.parametrize("name", ["x", "out_x", "out_n"])
@pytest.mark.parametrize("wrong", WRONG_ROWS, ids=str)
def test_forward_rows(group, name, wrong):
    assert _forward(group, **{name: _rows(**wrong)}) == BAD


def test_forward_rest(group):
    for name in ("y", "x", "w_pre", "out_x", "out_n"):
        assert _forward(group, **{name: None}) == BAD
    for v in WRONG_VECTORS:
        assert _forward(group, w_pre=v) == BAD
        assert _forward(group, w_post=v) == BAD
    assert _forward(group, gate=_rows(sizes=[2, H])) == BAD
    assert _forward(group, gate=_rows(dtype=A.EP_DTYPE_F32)) == BAD
    for f in (float("nan"), float("inf")):
        assert _forward(group, a=f) == BAD and _forward(group, b=f) == BAD and _forward(group, eps=f) == BAD
    assert _forward(group, eps=-1e-6) == BAD
    assert _forward(None) == BAD
    many = (1 << 22) + 1
    big = dict(sizes=[many, H])
    assert _forward(group, y=_rows(**big), x=_rows(**big), out_x=_rows(**big), out_n=_rows(**big)) == A.EP_ERR_UNSUPPORTED


def _backward(group, **over):
    t = dict(y=_rows(), x=_rows(), g_res=_rows(), g_norm=_rows(), w_post=_vec(), gate=None, w_pre=_vec(), d_res=_rows(),
             d_y=_rows(), d_pre=_vec(), d_post=_vec(), d_gate=None, work=_t(FAKE, A.EP_DTYPE_U8, [1 << 20]))
    t.update(over)
    return A.lib().ep_residual_norm_backward(
        group, _ref(t["y"]), _ref(t["x"]), _ref(t["g_res"]), _ref(t["g_norm"]), _ref(t["w_post"]), _ref(t["gate"]),
        _ref(t["w_pre"]), 1.0, 1.0, 1e-6, _ref(t["d_res"]), _ref(t["d_y"]), _ref(t["d_pre"]), _ref(t["d_post"]),
        _ref(t["d_gate"]), _ref(t["work"]), None)


@pytest.mark.parametrize("name", ["x", "g_res", "g_norm", "d_res", "d_y"])
@pytest.mark.parametrize("wrong", WRONG_ROWS, ids=str)
def test_backward_rows(group, name, wrong):
    assert _backward(group, **{name: _rows(**wrong)}) == BAD


def test_backward_rest(group):
    for name in ("y", "x", "g_norm", "w_pre", "d_res", "d_y", "d_pre", "work"):
        assert _backward(group, **{name: None}) == BAD
    for v in WRONG_VECTORS + [_vec(dtype=A.EP_DTYPE_BF16)]:
        assert _backward(group, d_pre=v) == BAD
        assert _backward(group, d_post=v) == BAD
    assert _backward(group, w_post=None) == BAD                       # a gradient of weights that are not there
    assert _backward(group, d_gate=_vec()) == BAD                     # of a gate that is not there
    one, each = _rows(sizes=[1, H]), _rows()
    assert _backward(group, gate=one, d_gate=_rows()) == BAD          # per channel: F32 [1, H]
    assert _backward(group, gate=each, d_gate=_vec()) == BAD          # per token: BF16 [n, H]
    need = ctypes.c_int64()
    assert A.lib().ep_residual_norm_workspace(group, N, ctypes.byref(need)) == A.EP_OK
    assert need.value >= 2 * N * H * 4
    assert _backward(group, work=_t(FAKE, A.EP_DTYPE_U8, [need.value - 1])) == BAD
    assert _backward(group, work=_t(FAKE + 4, A.EP_DTYPE_U8, [need.value])) == BAD
    assert _backward(group, work=_t(FAKE, A.EP_DTYPE_F32, [need.value])) == BAD
    assert A.lib().ep_residual_norm_workspace(group, -1, ctypes.byref(need)) == BAD
    assert A.lib().ep_residual_norm_workspace(None, 1, ctypes.byref(need)) == BAD
    assert A.lib().ep_residual_norm_workspace(group, 1, None) == BAD


def test_workspace_never_shrinks_below_its_use(group):
    """One share of two column sums per workgroup, at least as many bytes for more rows up to the full grid."""
    last = 0
    for n in (0, 1, 7, 255, 256, 257, 4096, 1 << 20):
        need = ctypes.c_int64()
        assert A.lib().ep_residual_norm_workspace(group, n, ctypes.byref(need)) == A.EP_OK
        assert need.value >= last and need.value % (2 * H * 4) == 0
        last = need.value


def test_products_reject_what_is_no_handle():
    lib = A.lib()
    junk = ctypes.addressof(ctypes.create_string_buffer(256))
    r, w = _rows(), _t(FAKE, A.EP_DTYPE_BF16, [256, 64, H])
    for h in (None, junk):
        assert lib.ep_expert_gated(h, _ref(r), _ref(w), _ref(w), None, None, 0, _ref(r), None) == BAD
        assert lib.ep_expert_gated_backward(h, _ref(r), _ref(w), _ref(w), _ref(r), 0, _ref(r), _ref(r), None, None, None,
                                            None) == BAD
        assert lib.ep_expert_quantize(h, _ref(r), _ref(r), _ref(r), None) == BAD
        assert lib.ep_expert_linear(h, _ref(r), None, _ref(w), None, _ref(r), None) == BAD
        assert lib.ep_expert_linear_backward(h, _ref(r), _ref(w), _ref(r), None, None, None) == BAD
