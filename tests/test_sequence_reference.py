"""The 64-bit plain forms of the sequence operators against closed forms and
differences (CPU)."""
import pytest
import torch

from tests import sequence_reference as R


def _inputs(gate, T=7, hk=1, hv=2, seqs=2):
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return [unit(rn(T, hk, 128)), unit(rn(T, hk, 128)), rn(T, hv, 128), torch.sigmoid(rn(T, hv)),
            torch.sigmoid(rn(*((T, hv) if gate == "gdn" else (T, hv, 128)))), 0.1 * rn(seqs * hv, 128, 128)]


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("delta", [True, False])
def test_gradient_against_differences(gate, delta):
    x = _inputs(gate)
    cu = [0, 3, 7]
    g = torch.Generator().manual_seed(6)
    wo = torch.randn((7, 2, 128), generator=g, dtype=torch.float64)
    ws = torch.randn((4, 128, 128), generator=g, dtype=torch.float64)

    def loss(args):
        o, S = R.recurrence(cu, *args, delta)
        return (o * wo).sum() + (S * ws).sum()

    leaves = [t.clone().requires_grad_(True) for t in x]
    grads = torch.autograd.grad(loss(leaves), leaves)
    h = 1e-6
    for n, (t, gr) in enumerate(zip(x, grads)):
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        hi, lo = ([y + s * h * d if m == n else y for m, y in enumerate(x)] for s in (1, -1))
        num = (loss(hi) - loss(lo)) / (2 * h)
        # truncation h^2 times third derivatives, rounding 2^-53 |loss| / h: both below 1e-8 of the sums here
        assert abs(num - (gr * d).sum()) <= 1e-6 * (gr * d).abs().sum(), n


def test_linear_attention_closed_form():
    q, k, v, beta, _, _ = _inputs("gdn", hk=2)
    one = torch.ones_like(beta)
    o, S = R.recurrence([0, 7], q, k, v, beta, one, torch.zeros(2, 128, 128, dtype=torch.float64), delta=False)
    want = torch.einsum("th,thi,thj->hij", beta, k, v)
    torch.testing.assert_close(S, want)
    torch.testing.assert_close(o[-1], torch.einsum("hij,hi->hj", want, q[-1]))


def test_delta_rule_writes_the_value():
    q, k, v, _, _, _ = _inputs("gdn", hk=2)
    one = torch.ones(7, 2, dtype=torch.float64)
    o, _ = R.recurrence([0, 7], k, k, v, one, one, torch.zeros(2, 128, 128, dtype=torch.float64))
    torch.testing.assert_close(o, v)  # a unit key with beta = 1 reads back what was just written


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_products_of_relative_positions(interleaved):
    g = torch.Generator().manual_seed(7)
    x, y = (torch.randn((1, 1, 128), generator=g, dtype=torch.float64) for _ in range(2))
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    dots = [(R.rotate(x, torch.tensor([p + 5]), f, interleaved) * R.rotate(y, torch.tensor([p]), f, interleaved)).sum()
            for p in (0, 1234, 99999)]
    torch.testing.assert_close(dots[1], dots[0])
    torch.testing.assert_close(dots[2], dots[0])
