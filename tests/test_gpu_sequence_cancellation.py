"""Results of the sequence operators that are small beside the terms they are
summed of: sums are fp32 whatever the type of the results, so an error counts
fp32 roundings of the terms, and one rounding of the result to its own type.

Keys of 64 entries of +-1/8 are exactly of unit norm in every type.  A token
of strength 1 whose query is its key then reads back the value it has just
written, o = v, whatever the state held: Gam (Q S0) and P U cancel.  With states
BIG times the values the terms are BIG times the result.

Bound (root mean squares; independent roundings, each uniform within 2^-24 of
a term, so 2^-24 / sqrt(3) of it).  On the chain of o stand Q S0 and K S0 (24
products of 32 terms and a sum of two each), T X and P U (12 and one each), the
inverse T (16 substitutions and 32 terms) and six single steps: n = 130.  A
gradient's chain holds that one, the reverse one (K G, P^T dO, T^T dU: 50) and
its own three products (80): n = 260.  Leaving out the third of three bf16
parts of the operands is 2^-19 of the terms, five times the bound of n = 130.
"""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import sequence_reference as R
from tests.test_gpu_sequence import BF16, DEV, F16, F32, GRADS, backward, forward, reference

pytestmark = pytest.mark.gpu
BIG = 2.0 ** 14


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def unit_keys(shape, g):
    """64 entries of +-1/8 in each row of 128."""
    pick = torch.rand((*shape, 128), generator=g).argsort(-1) < 64
    return torch.where(pick, (torch.randint(0, 2, (*shape, 128), generator=g) * 2 - 1) / 8.0, 0.0)


def rms(x):
    return float(x.double().square().mean().sqrt())


def allowed(ref, dtype, n, terms):
    """Root mean square that an error may have: of the rounding to dtype, and of n fp32 roundings of the terms."""
    own = R.step(dtype) / 3 ** 0.5 * rms(ref) if dtype != F32 else 0.0
    return own + (n / 3) ** 0.5 * R.U * terms


def overwritten(T, hk, hv, dtype, gate, seed):
    g = torch.Generator().manual_seed(seed)
    k = unit_keys((T, hk), g)
    # decays near 1: the states stay as large as they were
    decay = torch.rand((T, hv) if gate == "gdn" else (T, hv, 128), generator=g) * 2.0 ** -8
    return {"q": k.to(dtype), "k": k.to(dtype), "v": torch.randn((T, hv, 128), generator=g).to(dtype),
            "beta": torch.ones(T, hv), "alpha": 1 - decay}, g


# 6 tokens go token by token, 64 and 150 in chunks
@pytest.mark.parametrize("tokens", [6, 64, 150])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gate,save", [("gdn", False), ("gdn", True), ("kda", False)])
def test_overwritten_states_leave_the_values(gate, save, dtype, tokens):
    hk, hv = 1, 2
    x, g = overwritten(tokens, hk, hv, dtype, gate, 200 + tokens)
    x["S0"] = BIG * torch.randn((hv, 128, 128), generator=g)
    _, _, o, _ = forward([0, tokens], x, hk, hv, gate, save=save)
    off = o.double().cpu() - x["v"].double()
    # 52 roundings a chunk (K S0, T X and the update) that came before
    n = 130 + 52 * ((tokens - 1) // 64)
    assert rms(off) <= allowed(x["v"], dtype, n, BIG)


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_gradients_of_an_overwritten_state(dtype, delta):
    """One key for all tokens and a state of its direction alone: the first
    token replaces the whole state, so the later queries' and keys' gradients
    are small, and their terms with the state before it are not.  Without the
    delta correction a value of -w takes the state away."""
    T, hk, hv = 64, 1, 2
    x, g = overwritten(T, hk, hv, dtype, "gdn", 300)
    key = x["k"][0, 0].float()
    x["q"] = torch.where(torch.arange(T)[:, None, None] > 0, torch.randn((T, hk, 128), generator=g) * 128 ** -0.5,
                         x["q"].float()).to(dtype)
    x["k"] = x["k"][:1].expand(T, hk, 128).clone()
    w = (BIG * torch.randn((hv, 128), generator=g)).to(dtype)
    x["alpha"][:] = 1.0
    x["S0"] = key[None, :, None] * w.float()[:, None, :]
    if not delta:
        x["v"][0] = -w
    do = torch.randn((T, hv, 128), generator=g).to(dtype)
    do[0] = 0  # the first token's own gradients are large: they hold the state before it
    plan, d, _, _ = forward([0, T], x, hk, hv, "gdn", delta, save=True)
    got = backward(plan, [0, T], d, do.to(DEV))
    ref = dict(zip(GRADS, reference([0, T], x, delta, grads=(do, None))[2:]))
    # an entry of S0's rows is BIG / 8, a row of do times it sums 128 of them
    terms = BIG / 8 * 128 ** 0.5
    for m in ("q", "k"):
        r, y = ref[m][1:], got[m][1:].double().cpu()
        assert rms(r) < terms / 16, m  # (what the case is for)
        assert rms(y - r) <= allowed(r, dtype, 260, terms), m
