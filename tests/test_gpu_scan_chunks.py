"""The selective scan in chunks of 32 tokens and more, several of them a sequence,
as calls that fill the chip take them: every number of states, type, gate and
group count, against the 64-bit form on the device, all channels.

Roundings as counted in tests/layer_reference.py, but for the sums of the
gradients of B and C over the `per` channels of a group, which are counted as they
are made: four lanes in two additions, sixteen shares, then the waves of 64
channels one after another.  n = 9 T + 2 N + per / 64 + 184."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import scan_beside
from tests.sequence_reference import U, step

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
LOW = ("x", "dt", "B", "C", "z")

# Offsets (ends of chunks and of sequences that are no multiples of 8 or 4, tokens of no sequence around them),
# tokens and channels; tests/test_layer_rules.py holds the chunks of these calls to the lengths that are meant here:
# by the number of states, forward and of the gradient, whose chunks from zero are half as long
CU, TOKENS, CHANNELS = [2, 7, 7, 433, 1002], 1003, 8192
CHUNKS = {8: (48, 48), 16: (48, 72), 32: (48, 144)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def make(N, G, dtype, gate, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    T, c, n = TOKENS, CHANNELS, len(CU) - 1
    low = lambda *s: r(*s).to(dtype)  # noqa: E731
    return {"x": low(T, c), "dt": (0.5 * r(T, c)).to(dtype), "B": low(T, G, N), "C": low(T, G, N),
            "z": low(T, c) if gate else None, "dy": low(T, c), "A": -torch.arange(1, N + 1, device=DEV) * torch.exp(0.1 * r(c, N)),
            # steps of 0.01 to 0.5: what a chunk hands to the next is felt over most of it
            "D": 1 + 0.1 * r(c), "bias": 1.2 * r(c) - 3, "S0": r(n, c, N), "dS": r(n, c, N)}


def wide(t):
    return None if t is None else t.double()


def near(got, ref, n, name, mag):
    """Each entry within half a step of its type and n roundings of its own terms; and these bounds a small part of the
    values, so that what is lost shows: of 995 tokens and 128 waves a chunk of 48 tokens has the root of 48 / 995, 0.22, of
    a sum over tokens, a wave the root of 1 / 128, 0.088, of one over channels."""
    assert torch.isfinite(got).all(), name
    lim = n * U * mag * (1 + step(got.dtype)) + torch.finfo(F32).tiny
    assert lim.square().mean().sqrt() <= 0.08 * ref.square().mean().sqrt(), name
    if got.dtype != F32:
        lim = lim + ref.abs() * step(got.dtype) + torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    off = (got.double() - ref).abs()
    assert (off <= lim).all(), f"{name}: {int((off > lim).sum())} off, worst {float((off / lim).max()):.3g} times its bound"


@pytest.mark.parametrize("gate,G", [(True, 2), (False, 1), (True, 1), (False, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("N", [8, 16, 32])
def test_chunks_of_32_tokens_and_more(N, dtype, gate, G):
    d = make(N, G, dtype, gate, seed=N + 100 * G)
    cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
    n, c = len(CU) - 1, CHANNELS
    plan = lq.LeapQuantScan(TOKENS, n, c, N, groups=G, dtype=dtype, save=True)
    plan.workspace.fill_(255)  # NaN wherever it is read unwritten
    y, S = torch.full_like(d["x"], 7.0), torch.full_like(d["S0"], 7.0)
    kw = dict(D=d["D"], dt_bias=d["bias"], z=d["z"])
    lq.leapquant_scan_forward(plan, cu, d["x"], d["dt"], d["A"], d["B"], d["C"], y, S0=d["S0"], S=S, **kw)
    out = {m: torch.full_like(d[m], 7.0) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z", "S0") if d[m] is not None}
    lq.leapquant_scan_backward(plan, cu, d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], out["x"], out["dt"], out["A"],
                               out["B"], out["C"], dD=out["D"], ddt_bias=out["bias"], dz=out.get("z"), dS=d["dS"],
                               dS0=out["S0"], **kw)
    args = [wide(d[m]) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z", "S0", "dy", "dS")]
    ref, top = (scan_beside.scan_adjoint(CU, *args, absolute=a) for a in (False, True))
    keep = slice(CU[0], CU[-1])
    T = max(b - a for a, b in zip(CU, CU[1:]))
    near(y[keep], ref["y"][keep], 4 * T + N + 64, "y", top["y"][keep])
    near(S, ref["S"], 4 * T + 32, "S", top["S"])
    k = 9 * T + 2 * N + c // G // 64 + 184
    for m, t in out.items():
        if m in LOW:
            near(t[keep], ref[m][keep], k, "d" + m, top[m][keep])
        else:
            near(t, ref[m], k + (0 if m == "S0" else TOKENS), "d" + m, top[m])
    for t in (y, *(out[m] for m in LOW if m in out)):
        assert (t[:CU[0]] == 7).all() and (t[CU[-1]:] == 7).all()
    # without what is kept for the gradient
    plan = lq.LeapQuantScan(TOKENS, n, c, N, groups=G, dtype=dtype)
    plan.workspace.fill_(255)
    y2, S2 = torch.full_like(y, 7.0), torch.full_like(S, 7.0)
    lq.leapquant_scan_forward(plan, cu, d["x"], d["dt"], d["A"], d["B"], d["C"], y2, S0=d["S0"], S=S2, **kw)
    assert torch.equal(y, y2) and torch.equal(S, S2)
