"""The stream argument of the operators around the recurrence: their calls run on
that stream, not on the current one."""
import pytest
import torch

import recurrent_state_quant_amd as lq

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16
CU, T, C, N = [0, 150, 400], 400, 192, 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    low = lambda *s: r(*s).to(BF16)  # noqa: E731
    return dict(cu=torch.tensor(CU, dtype=torch.int32, device=DEV), x=low(T, C), dt=low(T, C) - 2, z=low(T, C), dy=low(T, C),
                B=low(T, 1, N), C=low(T, 1, N), A=-torch.exp(r(C, N)), w=r(C, 4), state=r(T, C, N), window=low(T, 3, C))


def conv(d, stream):
    y, dx, dw, X = torch.zeros_like(d["x"]), torch.zeros_like(d["x"]), torch.zeros_like(d["w"]), d["window"].clone()
    ws = lq.leapquant_conv_workspace(T, 2, C, 4)
    torch.cuda.synchronize()
    yield
    lq.leapquant_conv_forward(d["cu"], d["x"], d["w"], y, stream=stream)
    lq.leapquant_conv_backward(d["cu"], d["x"], d["w"], d["dy"], dx, dweight=dw, workspace=ws, stream=stream)
    lq.leapquant_conv_step(y, d["w"], dx, X, stream=stream)
    yield y, dx, dw, X


def scan(d, stream):
    plan = lq.LeapQuantScan(T, 2, C, N, save=True)
    y, g = torch.zeros_like(d["x"]), {m: torch.zeros_like(d[m]) for m in ("x", "dt", "A", "B", "C")}
    S = d["state"].clone()
    torch.cuda.synchronize()
    yield
    lq.leapquant_scan_forward(plan, d["cu"], d["x"], d["dt"], d["A"], d["B"], d["C"], y, stream=stream)
    lq.leapquant_scan_backward(plan, d["cu"], d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], g["x"], g["dt"], g["A"],
                               g["B"], g["C"], stream=stream)
    lq.leapquant_scan_step(y, d["dt"], d["A"], d["B"], d["C"], d["z"], S, stream=stream)
    yield y, *g.values(), d["z"], S


def norm(d, stream):
    row = lambda t: t.view(T, 1, C)  # noqa: E731
    h, y, da, dz = (torch.zeros_like(row(d["x"])) for _ in range(4))
    w = torch.ones(C, device=DEV)
    dw, ws = torch.zeros_like(w), lq.leapquant_block_norm_workspace(T, 1, C)
    torch.cuda.synchronize()
    yield
    lq.leapquant_block_norm(row(d["x"]), h=h, y=y, z=row(d["z"]), in_weight=w, stream=stream)
    lq.leapquant_block_norm_backward(row(d["x"]), da, dy=row(d["dy"]), z=row(d["z"]), dz=dz, in_weight=w, din_weight=dw,
                                     workspace=ws, stream=stream)
    yield h, y, da, dz, dw


@pytest.mark.parametrize("op", [conv, scan, norm])
def test_stream_argument(op):
    """The inputs become what they are on that stream, behind long work, and nothing else is waited for."""
    want = op(inputs(1), None)
    next(want)
    want = [t.clone() for t in next(want)]
    d, true = inputs(2), inputs(1)
    d["state"], d["window"] = true["state"], true["window"]  # copied ahead of the calls
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    call = op(d, side)
    next(call)
    with torch.cuda.stream(side):
        for _ in range(8):
            big = big @ big * 1e-2
        for m in d:
            d[m].copy_(true[m])
    got = next(call)
    side.synchronize()
    for k, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(a, b), k
