"""One long sequence among many short ones: few tokens a sequence on average,
so the whole call goes token by token; and the same batch in two calls, a form
each, on the same arrays."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests.test_gpu_sequence import BF16, DEV, F32, check_forward, forward, make, offsets, reference

pytestmark = pytest.mark.gpu
LENGTHS = [600] + [1, 1, 0, 1] * 12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 6)])  # up to 255 states, and more
@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_long_sequence_among_short_ones(gate, hk, hv, dtype):
    cu, x = make(LENGTHS, hk, hv, dtype, gate, seed=600, shift=3.0)
    _, _, o, S = forward(cu, x, hk, hv, gate)
    check_forward(cu, x, o, S, reference(cu, x))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_two_calls_on_the_same_arrays(gate):
    """Offsets of a part of the batch: its tokens and states alone are read and written."""
    hk, hv = 2, 4
    cu, x = make(LENGTHS, hk, hv, F32, gate, seed=601, shift=3.0)
    T, n = cu[-1], len(LENGTHS)
    d = {m: y.to(DEV) for m, y in x.items()}
    at = offsets(cu)
    o, S = torch.full((T, hv, 128), 7.0, device=DEV), torch.full_like(d["S0"], 7.0)
    plan = lq.LeapQuantSequence(T, n, hk, hv, gate, F32, DEV)
    names = ("q", "k", "v", "beta", "alpha")
    lq.leapquant_sequence_forward(plan, at[:2], *[d[m] for m in names], o, S0=d["S0"][:hv], S=S[:hv])
    assert (o[cu[1]:] == 7).all() and (S[hv:] == 7).all() and (o[:cu[1]] != 7).any()
    lq.leapquant_sequence_forward(plan, at[1:], *[d[m] for m in names], o, S0=d["S0"][hv:], S=S[hv:])
    check_forward(cu, x, o, S, reference(cu, x))
