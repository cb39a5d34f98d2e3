"""Outputs that lie head by head in one buffer: views whose ranges interleave
and whose elements do not."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import sequence_reference as R
from tests.test_gpu_sequence import BF16, DEV, F32, GRADS, check_backward, check_forward, make, offsets, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("major", ["tokens", "heads"])
@pytest.mark.parametrize("lengths", [[70, 20], [1]])
def test_gradients_interleaved_by_head(lengths, major):
    """dq, dk, dv in [tokens][heads][4][128] (a quarter left as it was) or its head-major form, the gates'
    gradients in [tokens][heads][2]; the inputs in a buffer of the same kind."""
    H, T = 2, sum(lengths)
    cu, x = make(lengths, H, H, F32, seed=400 + T)
    g = torch.Generator().manual_seed(401)
    do, dS = torch.randn(x["v"].shape, generator=g), torch.randn(x["S0"].shape, generator=g)

    def buffer():
        if major == "tokens":
            return torch.full((T, H, 4, 128), 7.0, device=DEV)
        return torch.full((H, T, 4, 128), 7.0, device=DEV).transpose(0, 1)

    ins, outs = buffer(), buffer()
    q, k, v, o = (ins[:, :, i] for i in range(4))
    for t, m in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(x[m])
    beta, alpha, S0 = (x[m].to(DEV) for m in ("beta", "alpha", "S0"))
    S = torch.empty_like(S0)
    plan = lq.LeapQuantSequence(T, len(lengths), H, H, dtype=F32, device=DEV, save=True)
    lq.leapquant_sequence_forward(plan, offsets(cu), q, k, v, beta, alpha, o, S0=S0, S=S)
    gates = torch.full((T, H, 2), 7.0, device=DEV)
    got = {"q": outs[:, :, 0], "k": outs[:, :, 1], "v": outs[:, :, 3], "beta": gates[..., 0], "alpha": gates[..., 1],
           "S0": torch.empty_like(S0)}
    lq.leapquant_sequence_backward(plan, offsets(cu), q, k, beta, alpha, do.to(DEV), *[got[m] for m in GRADS[:5]],
                                   dS=dS.to(DEV), dS0=got["S0"])
    ref = reference(cu, x, grads=(do, dS))
    check_forward(cu, x, o, S, ref[:2])
    check_backward(cu, got, ref[2:])
    assert (outs[:, :, 2] == 7).all()


def test_norm_outputs_interleaved_by_head():
    T, H = 33, 4
    g = torch.Generator().manual_seed(402)
    raw = torch.randn((T, 2 * H, 128), generator=g).to(BF16)
    out = torch.full((T, H, 2, 128), 7.0, device=DEV)
    lq.leapquant_head_norm(raw[:, :H].to(DEV), raw[:, H:].to(DEV), out[:, :, 0], out[:, :, 1])
    for i, x in enumerate((raw[:, :H], raw[:, H:])):
        R.check(out[:, :, i], R.head_norm(x.double(), "l2", 1e-6, None, 1.0, None, None, False), 160, "qk"[i])
