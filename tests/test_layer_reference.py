"""The 64-bit forms of the operators around the recurrence (CPU): their
gradients against differences, and the scan's written-out adjoint against
automatic differentiation."""
import pytest
import torch

from tests import layer_reference as R


def _rand(g, *s):
    return torch.randn(s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_conv_gradients(width, silu):
    g = torch.Generator().manual_seed(1)
    cu, c = [0, 3, 3, 5, 6], 2
    x, w, b, X0 = _rand(g, 6, c), _rand(g, c, width), _rand(g, c), _rand(g, 4, width - 1, c)
    leaves = [t.requires_grad_(True) for t in (x, w, b, X0)]
    assert torch.autograd.gradcheck(lambda *t: R.conv(cu, *t, silu)[:2], leaves)


def _scan_inputs(g, cu, c, N, G):
    T = cu[-1] + 1
    return [_rand(g, T, c), _rand(g, T, c) - 1, -torch.rand((c, N), generator=g, dtype=torch.float64) * 2,
            _rand(g, T, G, N), _rand(g, T, G, N), _rand(g, c), _rand(g, c), _rand(g, T, c), _rand(g, len(cu) - 1, c, N)]


@pytest.mark.parametrize("softplus", [False, True])
def test_scan_gradients(softplus):
    g = torch.Generator().manual_seed(2)
    cu = [1, 4, 4, 6]
    leaves = [t.requires_grad_(True) for t in _scan_inputs(g, cu, 4, 2, 2)]
    assert torch.autograd.gradcheck(lambda *t: R.scan(cu, *t, softplus=softplus), leaves)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("plain", [False, True])
def test_scan_adjoint(plain, softplus):
    """The formulas, also without a gate, a skip and a bias."""
    g = torch.Generator().manual_seed(3)
    cu = [0, 5, 5, 12, 13]
    v = _scan_inputs(g, cu, 6, 3, 2)
    if plain:
        v[5] = v[6] = v[7] = None
    names = ["x", "dt", "A", "B", "C", "D", "bias", "z", "S0"]
    leaves = [None if t is None else t.requires_grad_(True) for t in v]
    y, S = R.scan(cu, *leaves, softplus=softplus)
    dy, dS = _rand(g, *y.shape), _rand(g, *S.shape)
    ins = [(m, t) for m, t in zip(names, leaves) if t is not None]
    grads = torch.autograd.grad((y, S), [t for _, t in ins], (dy, dS))
    with torch.no_grad():
        r = R.scan_adjoint(cu, *leaves, dy, dS, softplus=softplus)
    assert torch.allclose(r["y"], y) and torch.allclose(r["S"], S)
    for (m, _), d in zip(ins, grads):
        assert torch.allclose(r[m], d, rtol=1e-9, atol=1e-11), m
    with torch.no_grad():
        top = R.scan_adjoint(cu, *leaves, dy, dS, softplus=softplus, absolute=True)
    for m in r:
        assert (top[m] >= r[m].abs() * (1 - 1e-12)).all(), m


@pytest.mark.parametrize("gate", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("out_norm", [False, True])
def test_block_norm_gradients(gate, out_norm):
    g = torch.Generator().manual_seed(4)
    a, res, wo, wi = _rand(g, 2, 1, 8), _rand(g, 2, 1, 8), _rand(g, 8), _rand(g, 8)
    z = None if gate == "none" else _rand(g, 2, 1, 8).requires_grad_(True)
    leaves = [t.requires_grad_(True) for t in (a, res, wo, wi)] + ([] if z is None else [z])

    def f(a, res, wo, wi, *z):
        return R.block_norm(a, z[0] if z else None, res, gate, 0.7, out_norm, wo if out_norm else None, wi, 1e-3)

    assert torch.autograd.gradcheck(f, leaves)
