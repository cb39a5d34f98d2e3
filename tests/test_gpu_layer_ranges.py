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
