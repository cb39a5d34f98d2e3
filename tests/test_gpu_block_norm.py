"""The norms before and after a block on the GPU against their 64-bit form.
Roundings are counted in tests/layer_reference.py: n = 2 dim + 64 forward, 4 dim +
128 for gradients, one more for each row in the weights'."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import layer_reference as R
from tests.sequence_reference import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def make(T, heads, dim, dtype, stream, gate, out_norm, res, weights, seed=0):
    g = torch.Generator().manual_seed(300 + seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    s = (T, heads, dim)
    x = {"a": r(*s).to(dtype), "z": r(*s).to(dtype) if gate != "none" else None, "res": (2 * r(*s)).to(stream) if res else None,
         "wo": 1 + 0.2 * r(dim) if weights and out_norm else None, "wi": 1 + 0.2 * r(dim) if weights else None,
         "dh": r(*s).to(stream), "dy": r(*s).to(dtype)}
    return x, dict(gate=gate, scale=0.37 if res else 1.0, out_norm=out_norm)


def dev(x):
    return {m: None if t is None else t.to(DEV) for m, t in x.items()}


def call(d, how, h=None, y=None):
    lq.leapquant_block_norm(d["a"], h=h, y=y, z=d["z"], res=d["res"], out_weight=d["wo"], in_weight=d["wi"], eps=EPS, **how)


def reference(x, how, use=("dh", "dy")):
    ins = {m: x[m].double().requires_grad_(True) for m in ("a", "z", "res", "wo", "wi") if x[m] is not None}
    get = ins.get
    h, y = R.block_norm(get("a"), get("z"), get("res"), how["gate"], how["scale"], how["out_norm"], get("wo"), get("wi"), EPS)
    outs = [t for t, m in ((h, "dh"), (y, "dy")) if m in use]
    grads = torch.autograd.grad(outs, list(ins.values()), [x[m].double() for m in use], materialize_grads=True)
    return h, y, dict(zip(ins, grads))


def backward(d, how, use=("dh", "dy"), dres=None):
    out = {m: torch.full_like(d[m], 7.0) for m in ("a", "z", "res", "wo", "wi") if d[m] is not None}
    if dres is not None:
        out["res"] = dres
    if "dy" not in use:
        out.pop("wi", None)
    T, heads, dim = d["a"].shape
    ws = lq.leapquant_block_norm_workspace(T, heads, dim)
    ws.fill_(255)
    lq.leapquant_block_norm_backward(d["a"], out["a"], dh=d["dh"] if "dh" in use else None, dy=d["dy"] if "dy" in use else None,
                                     z=d["z"], res=d["res"], out_weight=d["wo"], in_weight=d["wi"], eps=EPS, dz=out.get("z"),
                                     dres=out.get("res"), dout_weight=out.get("wo"), din_weight=out.get("wi"), workspace=ws,
                                     **how)
    return out


CASES = [(1, 1, 8, "silu", True, True, True), (3, 5, 128, "silu", True, False, True), (17, 2, 64, "sigmoid", True, True, False),
         (5, 1, 136, "none", False, True, True), (7, 1, 512, "silu", False, True, True), (9, 1, 1000, "none", True, True, True),
         (6, 1, 1032, "sigmoid", True, True, True), (5, 1, 2056, "silu", True, True, True), (4, 1, 4096, "none", False, True, True),
         (3, 1, 4104, "sigmoid", True, True, True), (2, 1, 8192, "silu", True, True, True), (70, 4, 128, "none", True, False, False),
         (33, 3, 256, "silu", False, False, True)]


@pytest.mark.parametrize("dtype,stream", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,heads,dim,gate,out_norm,res,weights", CASES)
def test_norm_and_gradient(T, heads, dim, gate, out_norm, res, weights, dtype, stream):
    x, how = make(T, heads, dim, dtype, stream, gate, out_norm, res, weights, seed=dim)
    d = dev(x)
    h_ref, y_ref, grads = reference(x, how)
    h, y = torch.empty((T, heads, dim), dtype=stream, device=DEV), torch.empty_like(d["a"])
    call(d, how, h, y)
    check(h, h_ref, 2 * dim + 64, "h")
    check(y, y_ref, 2 * dim + 64, "y")
    for one in ("h", "y"):  # one of them alone
        t = torch.empty_like(h if one == "h" else y)
        call(d, how, **{one: t}) if one == "h" or res is False or d["res"].dtype == stream else None
        assert torch.equal(t, h if one == "h" else y)
    out = backward(d, how)
    for m, g in grads.items():
        check(out[m], g, 4 * dim + 128 + (T * heads if m in ("wo", "wi") else 0), "d" + m)


@pytest.mark.parametrize("use", [("dh",), ("dy",)])
@pytest.mark.parametrize("T,heads,dim", [(5, 4, 128), (3, 1, 1000), (2, 1, 2048)])
def test_one_gradient_alone(T, heads, dim, use):
    x, how = make(T, heads, dim, F32, F32, "silu", True, True, True, seed=1)
    d = dev(x)
    _, _, grads = reference(x, how, use)
    out = backward(d, how, use)
    for m in out:
        check(out[m], grads[m], 4 * dim + 128 + (T * heads if m in ("wo", "wi") else 0), "d" + m)


def test_many_rows():
    """More rows than the workgroups of the backward pass take at once."""
    for T, heads, dim in ((3000, 16, 64), (5001, 1, 264), (2100, 1, 1536)):
        x, how = make(T, heads, dim, F32, F32, "silu", True, True, True, seed=2)
        d = dev(x)
        w = {m: d[m] for m in x}
        ins = {m: w[m].double().requires_grad_(True) for m in ("a", "z", "res", "wo", "wi")}
        h, y = R.block_norm(ins["a"], ins["z"], ins["res"], "silu", how["scale"], True, ins["wo"], ins["wi"], EPS)
        grads = dict(zip(ins, torch.autograd.grad((h, y), list(ins.values()), (d["dh"].double(), d["dy"].double()))))
        out = backward(d, how)
        for m, g in grads.items():
            check(out[m], g, 4 * dim + 128 + (T * heads if m in ("wo", "wi") else 0), "d" + m)
        again = backward(d, how)
        assert all(torch.equal(out[m], again[m]) for m in out)


def test_in_place():
    """h over res, y over a, the stream's gradient over itself: the same results."""
    for T, heads, dim in ((40, 3, 128), (9, 1, 600), (5, 1, 3000), (3, 1, 6000)):
        x, how = make(T, heads, dim, BF16, F32, "silu", True, True, True, seed=3)
        d = dev(x)
        h, y = torch.empty_like(d["res"]), torch.empty_like(d["a"])
        call(d, how, h, y)
        over = {**d, "res": d["res"].clone(), "a": d["a"].clone()}
        call(over, how, over["res"], over["a"])
        assert torch.equal(over["res"], h) and torch.equal(over["a"], y)
        first = backward(d, how)
        dh = d["dh"].clone()
        second = backward({**d, "dh": dh}, how, dres=dh)
        assert all(torch.equal(first[m], second[m]) for m in first)
    # the gated norm of heads, over its input
    x, how = make(30, 8, 128, BF16, BF16, "silu", True, False, True, seed=4)
    d = dev(x)
    h, a = torch.empty_like(d["a"]), d["a"].clone()
    call(d, how, h)
    call({**d, "a": a}, how, a)
    assert torch.equal(a, h)


def test_slices_and_head_major():
    """Slices of wider rows and arrays that lie head by head; the memory between is left as it is."""
    x, how = make(20, 4, 128, F16, F16, "silu", True, False, True, seed=5)
    d = dev(x)
    h = torch.empty_like(d["a"])
    call(d, how, h)
    big = torch.full((20, 12, 136), 9.0, dtype=F16, device=DEV)
    a, z = big[:, 1:5, :128], big[:, 6:10, 8:]
    a.copy_(d["a"])
    z.copy_(d["z"])
    out = torch.full((4, 21, 128), 9.0, dtype=F16, device=DEV)
    call({**d, "a": a, "z": z}, how, out[:, :20].transpose(0, 1))
    assert torch.equal(out[:, :20].transpose(0, 1), h) and (out[:, 20] == 9).all()


def test_zero_rows_and_values_that_are_not_finite():
    """A row of zeros gives zeros and finite gradients; others are untouched by a row that is not finite."""
    for T, heads, dim in ((20, 2, 128), (6, 1, 520), (5, 1, 1200)):
        x, how = make(T, heads, dim, F32, F32, "silu", True, True, True, seed=6)
        x["a"][1], x["res"][1] = 0.0, 0.0
        d = dev(x)
        h, y = torch.empty_like(d["a"]), torch.empty_like(d["a"])
        call(d, how, h, y)
        assert (h[1] == 0).all() and (y[1] == 0).all()
        g = backward(d, how)
        assert all(torch.isfinite(t).all() for t in g.values())
        x["a"][2, 0, 3], x["dy"][3, 0, 5] = float("nan"), float("inf")
        d = dev(x)
        h2, y2 = torch.empty_like(h), torch.empty_like(y)
        call(d, how, h2, y2)
        g2 = backward(d, how)
        rows = torch.ones((T, heads), dtype=torch.bool, device=DEV)
        rows[2, 0] = rows[3, 0] = False
        assert torch.equal(h[rows], h2[rows]) and torch.equal(y[rows], y2[rows])
        for m in ("a", "z", "res"):
            assert torch.equal(g[m][rows], g2[m][rows]), m


def test_no_rows():
    a = torch.empty((0, 4, 128), device=DEV)
    lq.leapquant_block_norm(a, h=torch.empty_like(a), out_norm=True)
    dw = torch.full((128,), 7.0, device=DEV)
    lq.leapquant_block_norm_backward(a, torch.empty_like(a), dh=a, out_norm=True, dout_weight=dw)
    assert (dw == 0).all()


def test_far_offsets():
    """Element offsets beyond 2^31."""
    x, how = make(600, 1, 64, BF16, BF16, "none", True, False, True, seed=7)
    d = dev(x)
    h = torch.empty_like(d["a"])
    call(d, how, h)
    stride = 4_000_000
    far = lambda: torch.empty(600 * stride, dtype=BF16, device=DEV).as_strided((600, 1, 64), (stride, 64, 1))  # noqa: E731
    a, out = far(), far()
    a.copy_(d["a"])
    call({**d, "a": a}, how, out)
    assert torch.equal(out, h)


def test_captured_call():
    x, how = make(33, 1, 2048, BF16, F32, "sigmoid", True, True, True, seed=8)
    d = dev(x)
    res, a = d["res"].clone(), d["a"].clone()
    h, y = torch.empty_like(res), torch.empty_like(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = {**d, "res": res, "a": a}
    with torch.cuda.stream(side):
        call(s, how, h, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(s, how, h, y)
    torch.cuda.synchronize()
    for k in range(4):
        a.copy_((d["a"] * (k + 1)).to(BF16))
        graph.replay()
        h2, y2 = torch.empty_like(h), torch.empty_like(y)
        call(s, how, h2, y2)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(y, y2)


def test_refusals_on_the_device():
    z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    a = z(4, 2, 64)
    ok = dict(h=z(4, 2, 64), y=z(4, 2, 64), z=z(4, 2, 64), res=z(4, 2, 64))
    lq.leapquant_block_norm(a, **ok)
    for kw in (dict(h=z(4, 2, 32)), dict(y=z(4, 2, 64).half()), dict(z=z(4, 2, 64).cpu()), dict(res=z(4, 64, 2).transpose(1, 2)),
               dict(h=z(4, 2, 64).half()), dict(in_weight=z(32)), dict(in_weight=z(64).half())):
        with pytest.raises((ValueError, TypeError)):
            lq.leapquant_block_norm(a, **{**ok, **kw})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_block_norm(a, **{**ok, "y": ok["h"]})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_block_norm(z(4, 2, 12), h=z(4, 2, 12))
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_block_norm_backward(a, z(4, 2, 64), dh=a, out_norm=True, dout_weight=z(64))
