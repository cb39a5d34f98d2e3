"""Gradients of the sequence operators against central differences of the loss
along the gradient itself, where the derivative is as large as it can be.

x is moved by +-h v, v = g |x| / |g|: the difference's slope is to be g . v = |g| |x|.
With h = 2^-7 its truncation is h^2 / 6 = 1e-5 of the third derivative along v;
the loss is of third order in a key at most times a token, and its rounding
(2^-24 sqrt(130 / 3) of its terms, 2^6 / h times in a slope) is 5e-5 of them:
1e-3 of the slope is allowed for both.  A gradient that is scaled, negated or
in another order fails: the slope is the true gradient's along v.
"""
import pytest
import torch

from tests import sequence_reference as R

GRADS = ("q", "k", "v", "beta", "alpha", "S0")
H, TOLERANCE = 2.0 ** -7, 1e-3
CU, HK, HV = [0, 80, 100], 1, 2


def inputs():
    """fp32 inputs whose decays and strengths stay between 0 and 1 when they are moved, and the loss's weights."""
    g = torch.Generator().manual_seed(520)
    T, n = CU[-1], (len(CU) - 1) * HV
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(torch.randn((T, HK, 128), generator=g)), "k": unit(torch.randn((T, HK, 128), generator=g)),
         "v": torch.randn((T, HV, 128), generator=g), "beta": 0.25 + 0.5 * torch.rand((T, HV), generator=g),
         "alpha": 0.45 + 0.4 * torch.rand((T, HV), generator=g), "S0": 0.1 * torch.randn((n, 128, 128), generator=g)}
    return x, torch.randn((T, HV, 128), generator=g), 0.1 * torch.randn((n, 128, 128), generator=g)


def slopes(loss, x, m, grad):
    """(slope of the loss along grad, the gradient's own), with the inputs' rounding taken into account."""
    grad = grad.detach().double().cpu()
    v = grad * (x[m].double().norm() / grad.norm())
    hi, lo = ((x[m].double() + s * H * v).float() for s in (1, -1))
    if m in ("beta", "alpha"):
        assert min(float(lo.min()), float(hi.min())) >= 0 and max(float(lo.max()), float(hi.max())) <= 1
    num = (loss({**x, m: hi}) - loss({**x, m: lo})) / (2 * H)
    return float(num), float((grad * (hi.double() - lo.double())).sum() / (2 * H))


def agree(num, own):
    return abs(num - own) <= TOLERANCE * abs(own)


def _reference():
    x, do, dS = inputs()

    def loss(y):
        o, S = R.recurrence(CU, *[y[m].double() for m in GRADS])
        return (o * do.double()).sum() + (S * dS.double()).sum()

    leaves = {m: y.double().requires_grad_(True) for m, y in x.items()}
    grads = torch.autograd.grad(loss(leaves), [leaves[m] for m in GRADS])
    return x, loss, dict(zip(GRADS, grads))


def test_reference_agrees_and_wrong_gradients_do_not():
    x, loss, grads = _reference()
    g = torch.Generator().manual_seed(521)
    for m in GRADS:
        right = grads[m].detach()
        num, own = slopes(loss, x, m, right)
        assert abs(num - own) <= TOLERANCE / 10 * abs(own), (m, num, own)  # the truncation leaves room for rounding
        order = torch.randperm(right.numel(), generator=g)
        for wrong in (1.01 * right, 10 * right, -right, right.flatten()[order].view(right.shape)):
            assert not agree(*slopes(loss, x, m, wrong)), m


@pytest.mark.gpu
def test_gradients_along_themselves():
    from tests.test_gpu_sequence import DEV, backward, forward
    x, do, dS = inputs()
    plan, d, _, _ = forward(CU, x, HK, HV, save=True)
    grads = backward(plan, CU, d, do.to(DEV), dS.to(DEV))

    def loss(y):
        _, _, o, S = forward(CU, y, HK, HV)
        return (o.double().cpu() * do.double()).sum() + (S.double().cpu() * dS.double()).sum()

    for m in GRADS:
        num, own = slopes(loss, x, m, grads[m])
        assert agree(num, own), (m, num, own)
