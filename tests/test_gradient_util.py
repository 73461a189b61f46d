"""What the comparison of gradients with differences notices, on a 64-bit gated block (CPU): the right gradients pass
at the tolerances that the GPU tests use, rounded to bf16 too; a flipped sign, noise of the same norm, a gradient a
tenth too large, another expert's, an expert left out and a dropped term of the adjoint do not."""
import pytest
import torch

from gradient_util import D, check, mismatch

E, R, H, I = 3, 6, 64, 40
HALF = 2.0 ** -8
DELTA = 10 * HALF   # the widest that the GPU tests use


def block(x, wg, wu, wd):
    out = []
    for e in range(E):
        g, u = x[e] @ wg[e].t(), x[e] @ wu[e].t()
        out.append((g * torch.sigmoid(g) * u) @ wd[e].t())
    return torch.stack(out)


@pytest.fixture(scope="module")
def case():
    gen = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, dtype=D) * shape[-1] ** -0.5 * 2
    leaves = [normal(E, R, H).requires_grad_(), normal(E, I, H).requires_grad_(), normal(E, I, H).requires_grad_(),
              normal(E, H, I).requires_grad_()]
    up = torch.randn((E, R, H), generator=gen, dtype=D)
    (block(*leaves) * up).sum().backward()
    point = [t.detach() for t in leaves]
    losses = [lambda t, k=k: float((block(*point[:k], t, *point[k + 1:]) * up).sum()) for k in range(4)]
    return point, [t.grad for t in leaves], losses, up


@pytest.mark.parametrize("k", range(4), ids=["rows", "gate", "up", "down"])
def test_right_and_wrong_gradients(case, k):
    point, grads, losses, _ = case
    g, loss, x = grads[k], losses[k], point[k]
    check(g, g, loss, x, 2.0 ** -20, "exact")
    check(g.to(torch.bfloat16), g, loss, x, 2 * HALF, "bf16")
    noise = torch.randn(g.shape, generator=torch.Generator().manual_seed(5), dtype=D)
    wrong = {"sign": -g, "noise": noise * g.norm() / noise.norm(), "larger": 1.1 * g, "another expert's": g.roll(1, 0),
             "one left out": g * (torch.arange(E) > 0)[:, None, None]}
    for what, w in wrong.items():
        assert mismatch(w, g, loss, x, DELTA) is not None, what


def test_wrong_reference_does_not_hide_it(case):
    """The same mistake in the gradient and in the reference: seen along the gradient itself."""
    point, grads, losses, _ = case
    for k in range(4):
        assert mismatch(-grads[k], -grads[k], losses[k], point[k], DELTA) is not None
        assert mismatch(1.1 * grads[k], 1.1 * grads[k], losses[k], point[k], DELTA) is not None


def test_dropped_term(case):
    """act' without its second part, s(g) alone for s + g s (1 - s): a plausible mistake in the adjoint."""
    point, grads, losses, up = case
    x, wg, wu, wd = point
    w = []
    for e in range(E):
        g, u, da = x[e] @ wg[e].t(), x[e] @ wu[e].t(), up[e] @ wd[e]
        w.append((da * u * torch.sigmoid(g)).t() @ x[e])
    assert mismatch(torch.stack(w), grads[1], losses[1], wg, DELTA) is not None
