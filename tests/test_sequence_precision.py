"""The precision that fp32 results of the sequence operators keep: root mean
squares of their errors against 64 bits, in fp32 roundings of the results'
own (2^-24 / sqrt(3) each; the inputs are such that terms do not cancel).

On the chain of o and S stand n = 130 roundings in a sequence's first chunk (Q S0
and K S0: 24 products of 32 terms and a sum of two each; T X and P U: 12 and one
each; the inverse T: 16 substitutions and 32 terms; six single steps) and 52
(K S0, T X, the update) for each later one; on a gradient's another 130 (the
reverse chain and its own three products); on dbeta's and dalpha's 100 more (sums
along 128 values, running products of 64 decays and of the gradients behind them).
Independent roundings add up as sqrt(n).  Operands without their third bf16
part are off by 50 to 230 units of 2^-24 (the first test), five times the bounds.
"""
import pytest
import torch

from tests import sequence_parts, sequence_reference as R

NAMES = ("o", "S", "dq", "dk", "dv", "dbeta", "dalpha", "dS0")


def rms(x):
    return float(x.double().square().mean().sqrt())


def roundings(name, tokens):
    n = 130 + 52 * (max(tokens - 1, 0) // 64)
    if name in ("o", "S"):
        return n
    return n + (230 if name in ("dbeta", "dalpha") else 130)


def excess(got, ref, name, tokens):
    """The error's root mean square beside what it may be."""
    return rms(got.double().cpu() - ref.double().cpu()) / ((roundings(name, tokens) / 3) ** 0.5 * R.U * rms(ref))


def inputs(lengths, hk, hv, seed, shift, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    T, n = sum(lengths), len(lengths) * hv
    x = {"q": unit(rn(T, hk, 128)).to(dtype), "k": unit(rn(T, hk, 128)).to(dtype), "v": rn(T, hv, 128).to(dtype),
         "beta": torch.sigmoid(rn(T, hv)), "alpha": torch.exp(-torch.nn.functional.softplus(rn(T, hv) - shift)),
         "S0": 0.1 * rn(n, 128, 128)}
    return x, rn(T, hv, 128).to(dtype), 0.1 * rn(n, 128, 128)


def reference(lengths, x, do, dS, dev="cpu"):
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    leaves = [x[m].double().to(dev).requires_grad_(True) for m in ("q", "k", "v", "beta", "alpha", "S0")]
    o, S = R.recurrence(cu, *leaves)
    loss = (o * do.double().to(dev)).sum() + (S * dS.double().to(dev)).sum()
    return cu, dict(zip(NAMES, (o.detach(), S.detach(), *torch.autograd.grad(loss, leaves))))


@pytest.mark.parametrize("tokens,shift", [(20, 0.0), (64, 0.0), (200, 4.0)])
def test_dropped_parts_are_outside_the_bounds(tokens, shift):
    x, do, dS = inputs([tokens], 1, 1, 530 + tokens, shift)
    _, ref = reference([tokens], x, do, dS)
    one = [x[m][:, 0] for m in ("q", "k", "v", "beta", "alpha")] + [x["S0"][0], do[:, 0], dS[0]]
    for parts in (3, 2):
        got = dict(zip(NAMES, sequence_parts.forward_backward(*one, parts)))
        for m in NAMES:
            e = excess(got[m], ref[m].view(got[m].shape), m, tokens)
            assert (e <= 1) if parts == 3 else (e > 1), (m, parts, e)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lengths,hk,hv,shift", [([20], 1, 2, 0.0), ([64], 2, 2, 4.0), ([200, 130, 64], 2, 4, 4.0),
                                                 ([500, 333], 1, 4, 4.0), ([70] * 33, 1, 4, 2.0)])
def test_fp32_results_keep_their_precision(lengths, hk, hv, shift, dtype):
    """All results in fp32; of 16-bit inputs those that are fp32 all the same."""
    from tests.test_gpu_sequence import DEV, backward, forward
    x, do, dS = inputs(lengths, hk, hv, 540 + len(lengths), shift, dtype)
    cu, ref = reference(lengths, x, do, dS, DEV)
    plan, d, o, S = forward(cu, x, hk, hv, save=True)
    g = backward(plan, cu, d, do.to(DEV), dS.to(DEV))
    got = {"o": o, "S": S, **{"d" + m: y for m, y in g.items()}}
    _, _, o1, S1 = forward(cu, x, hk, hv)
    off = {m: excess(got[m], ref[m], m, max(lengths)) for m in NAMES if got[m].dtype == torch.float32}
    for m, y in (("o", o1), ("S", S1)):
        if y.dtype == torch.float32:
            off[m + " alone"] = excess(y, ref[m], m, max(lengths))
    print({m: round(e, 3) for m, e in off.items()})
    assert all(e <= 1 for e in off.values()), off


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,hk,hv,shift", [([20], 1, 2, 0.0), ([90, 64], 2, 4, 0.0), ([400, 3], 1, 2, 4.0)])
def test_fp32_results_with_a_decay_a_channel(lengths, hk, hv, shift):
    """As above, with 80 roundings more: products of 64 and 16 decays for every operand."""
    from tests.test_gpu_sequence import DEV, forward
    x, _, _ = inputs(lengths, hk, hv, 560 + len(lengths), shift)
    g = torch.Generator().manual_seed(561)
    x["alpha"] = torch.exp(-torch.nn.functional.softplus(torch.randn((sum(lengths), hv, 128), generator=g) - shift))
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    ref = R.recurrence(cu, *[x[m].double().to(DEV) for m in ("q", "k", "v", "beta", "alpha", "S0")])
    _, _, o, S = forward(cu, x, hk, hv, "kda")
    for name, y, r in (("o", o, ref[0]), ("S", S, ref[1])):
        n = roundings(name, max(lengths)) + 80
        assert rms(y.double() - r) <= (n / 3) ** 0.5 * R.U * rms(r), name
