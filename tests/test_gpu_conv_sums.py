"""The convolution's sums over many tokens, and the runs that many channels take,
against the 64-bit form on the device.

A weight's gradient is summed over the tokens of a run one after another, over
four runs in three additions, and over the blocks of four runs one after another:
n = 64 (layer_reference: what a token's term is off by) + run + 4 + blocks
roundings of the sum of its own terms' absolute values."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests.sequence_reference import U, check, step

pytestmark = pytest.mark.gpu
DEV, K = "cuda", 4
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# Tokens, channels, type; the forward run, the gradient's, and its blocks of four runs, to which
# tests/test_layer_rules.py holds these calls
CASES = [(8192, 8, F32, 32, 32, 64), (33000, 8, F32, 32, 64, 129), (66_001, 8, BF16, 32, 128, 129),
         (16500, 4096, F32, 64, 64, 65), (16384, 8192, BF16, 64, 64, 64), (16401, 8192, F16, 64, 64, 65),
         (8192, 6144, BF16, 32, 64, 32)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def exact(cu, v):
    """y, X and the gradients in 64 bits, and the sums of the absolute terms of y's v and of the weights' gradients."""
    rows, ys, lasts, mags = [], [], [], []
    dw, db, mw, mb = (torch.zeros_like(t) for t in (v["w"], v["b"], v["w"], v["b"]))
    dx, dX0 = [], []
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        n = hi - lo
        row = torch.cat((v["X0"][i], v["x"][lo:hi]))
        terms = [row[j:j + n] * v["w"][:, j] for j in range(K)]
        pre = sum(terms) + v["b"]
        s = torch.sigmoid(pre)
        ys.append(pre * s)
        mags.append(sum(t.abs() for t in terms) + v["b"].abs())
        lasts.append(row[n:])
        g = v["dy"][lo:hi] * (s * (1 + pre * (1 - s)))
        most = 1.1 * v["dy"][lo:hi].abs()
        drow = torch.zeros_like(row)
        drow[n:] = v["dX"][i]
        for j in range(K):
            drow[j:j + n] += g * v["w"][:, j]
            dw[:, j] += (g * row[j:j + n]).sum(0)
            mw[:, j] += (most * row[j:j + n].abs()).sum(0)
        db += g.sum(0)
        mb += most.sum(0)
        dx.append(drow[K - 1:])
        dX0.append(drow[:K - 1])
    return (torch.cat(ys), torch.stack(lasts), torch.cat(mags),
            {"x": torch.cat(dx), "X0": torch.stack(dX0), "w": dw, "b": db}, {"w": mw, "b": mb})


@pytest.mark.parametrize("tokens,c,dtype,run,run_grad,blocks", CASES)
def test_many_runs(tokens, c, dtype, run, run_grad, blocks):
    cu = [0, 1, 3, 3, tokens // 3, tokens - 40, tokens]
    g = torch.Generator(device=DEV).manual_seed(tokens + c)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    seqs = len(cu) - 1
    d = {"x": r(tokens, c).to(dtype), "w": 0.5 * r(c, K), "b": 0.3 * r(c), "X0": r(seqs, K - 1, c).to(dtype),
         "dy": r(tokens, c).to(dtype), "dX": r(seqs, K - 1, c).to(dtype)}
    where = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y, X = torch.full_like(d["x"], 7.0), torch.full_like(d["X0"], 7.0)
    lq.leapquant_conv_forward(where, d["x"], d["w"], y, bias=d["b"], X0=d["X0"], X=X)
    out = {m: torch.full_like(d[m], 7.0) for m in ("x", "w", "b", "X0")}
    ws = lq.leapquant_conv_workspace(tokens, seqs, c, K)
    ws.fill_(255)  # NaN wherever it is read unwritten
    lq.leapquant_conv_backward(where, d["x"], d["w"], d["dy"], out["x"], bias=d["b"], X0=d["X0"], dweight=out["w"],
                               dbias=out["b"], dX=d["dX"], dX0=out["X0"], workspace=ws)
    # up to 64 channels, of every lane and of every tile
    pick = torch.arange(c, device=DEV) if c <= 64 else (torch.arange(64, device=DEV) * (c // 64 + 1)) % c
    axis = {"x": 1, "w": 0, "b": 0, "X0": 2, "dy": 1, "dX": 2}
    some = lambda m, t: t.index_select(axis[m], pick)  # noqa: E731
    y64, X64, mag, grads, mags = exact(cu, {m: some(m, t).double() for m, t in d.items()})
    assert mag.max() <= 16
    check(some("x", y), y64, 16, "y", mag)
    assert torch.equal(some("X0", X).double(), X64)
    top = torch.tensor(1.1 * float(d["dy"].abs().max()) * 4 * float(d["w"].abs().max()) + float(d["dX"].abs().max()))
    check(some("x", out["x"]), grads["x"], 64, "dx", top)
    check(some("X0", out["X0"]), grads["X0"], 64, "dX0", top)
    for m in ("w", "b"):
        lim = (64 + run_grad + 4 + blocks) * U * mags[m]
        # (a run that is lost or counted twice moves a sum by about the root of its tokens)
        assert lim.max() <= 0.2 * run_grad ** 0.5
        assert ((some(m, out[m]).double() - grads[m]).abs() <= lim).all(), m
