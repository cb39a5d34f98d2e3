"""The operators around the recurrence at the ends of their inputs' ranges."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import layer_reference as R
from tests.sequence_reference import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("of", [1.0, 2.0 ** 47])  # (below 2^50: five standard deviations)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [128, 136, 512, 1024, 2048, 4096, 8192])
def test_norms_of_the_largest_values(dim, dtype, of):
    """Rows of values next to 2^60, whose squares sum to 2^133 in the widest: outputs and gradients of the norm of the
    block and of the stream.  Roundings as in tests/layer_reference.py."""
    g = torch.Generator().manual_seed(dim)
    T, top, eps = 3, 2.0 ** 60, 1e-5
    sign = lambda: 2.0 * (torch.rand((T, 1, dim), generator=g) < 0.5) - 1  # noqa: E731
    large = lambda: (sign() * top * (0.9 + 0.09 * torch.rand((T, 1, dim), generator=g))).to(dtype)  # noqa: E731
    for out_norm in (True, False):
        # normed values join a stream of large ones, or large ones a small stream
        a, res = large(), (large() if out_norm else torch.randn((T, 1, dim), generator=g).to(dtype))
        wo, wi = (1 + 0.2 * torch.randn(dim, generator=g) for _ in range(2))
        dh, dy = ((of * torch.randn((T, 1, dim), generator=g)).to(dtype) for _ in range(2))
        how = dict(scale=1.0, out_norm=out_norm, eps=eps)
        leaves = [t.double().requires_grad_(True) for t in (a, res, wo, wi)]
        h64, y64 = R.block_norm(leaves[0], None, leaves[1], "none", 1.0, out_norm, leaves[2] if out_norm else None,
                                leaves[3], eps)
        grads = torch.autograd.grad((h64, y64), leaves, (dh.double(), dy.double()), materialize_grads=True)
        d = [t.to(DEV) for t in (a, res, wo, wi, dh, dy)]
        h, y, da, dres = (torch.empty_like(d[0]) for _ in range(4))
        dwo, dwi = torch.empty_like(d[2]), torch.empty_like(d[3])
        kw = dict(res=d[1], out_weight=d[2] if out_norm else None, in_weight=d[3], **how)
        lq.leapquant_block_norm(d[0], h=h, y=y, **kw)
        check(h, h64, 2 * dim + 64, "h")
        check(y, y64, 2 * dim + 64, "y")
        assert y.abs().max() > 0.5
        lq.leapquant_block_norm_backward(d[0], da, dh=d[4], dy=d[5], dres=dres, dout_weight=dwo if out_norm else None,
                                         din_weight=dwi, workspace=lq.leapquant_block_norm_workspace(T, 1, dim), **kw)
        check(da, grads[0], 4 * dim + 128, "da")
        check(dres, grads[1], 4 * dim + 128, "dres")
        if out_norm:
            check(dwo, grads[2], 4 * dim + 128 + T, "dwo")
        check(dwi, grads[3], 4 * dim + 128 + T, "dwi")


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("v", [-60.0, -24.0, -12.0, -7.0, -3.0, 3.0, 12.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_steps_of_16_bit_inputs(dtype, v, bias):
    """Their states and the fp32 gradients keep the accuracy of fp32 sums: a step log(1 + e^v) is off by the 16
    roundings of tests/layer_reference.py and by three of |v|: the sum of dt and its bias, the exponent's product with
    log2 e (of which calls with 16-bit inputs leave the rest out) and log2 e itself, a quarter."""
    cu, c, N = [0, 1, 3], 64, 8
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x = {m: r(3, c).to(dtype) for m in ("x", "dy")} | {m: r(3, 1, N).to(dtype) for m in ("B", "C")}
    x["dt"] = (0.3 * r(3, c) if bias else v * (1 + 0.1 * torch.rand((3, c), generator=g))).to(dtype)
    x["A"], x["bias"] = -torch.rand((c, N), generator=g) - 0.1, v + 0.1 * r(c) if bias else None
    far = float((x["dt"].float() + (0 if x["bias"] is None else x["bias"])).abs().max())
    d = {m: None if t is None else t.to(DEV) for m, t in x.items()}
    plan = lq.LeapQuantScan(3, 2, c, N, dtype=dtype, save=True)
    where = torch.tensor(cu, dtype=torch.int32, device=DEV)
    y, S = torch.empty_like(d["x"]), torch.empty((2, c, N), device=DEV)
    lq.leapquant_scan_forward(plan, where, d["x"], d["dt"], d["A"], d["B"], d["C"], y, dt_bias=d["bias"], S=S)
    out = {m: torch.empty_like(d[m]) for m in ("x", "dt", "A", "B", "C")}
    db = None if x["bias"] is None else torch.empty_like(d["bias"])
    lq.leapquant_scan_backward(plan, where, d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], out["x"], out["dt"], out["A"],
                               out["B"], out["C"], dt_bias=d["bias"], ddt_bias=db)
    w = {m: None if t is None else t.double() for m, t in x.items()}
    zero = torch.zeros((2, c, N), dtype=torch.float64)
    args = [w["x"], w["dt"], w["A"], w["B"], w["C"], None, w["bias"], None, zero, w["dy"], zero]
    ref, top = (R.scan_adjoint(cu, *args, absolute=a) for a in (False, True))
    # of each entry's own terms; a gradient of A has two steps in a term, a step's slope is off by as much as the step
    for got, m, n in ((S, "S", 4 * 2 + 32 + 3 * far), (out["A"], "A", 9 * 2 + 2 * N + c + 160 + 3 + 6 * far),
                      (db, "bias", 9 * 2 + 2 * N + c + 160 + 3 + 6 * far)):
        if got is not None:
            off = (got.cpu().double() - ref[m]).abs()
            assert (off <= n * 2.0 ** -24 * top[m] + 2.0 ** -120).all(), m
