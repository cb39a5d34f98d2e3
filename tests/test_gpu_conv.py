"""The short causal convolution on the GPU against its 64-bit form.  Roundings
counted in tests/layer_reference.py: n = 16 for a value, 64 for a gradient, one
more for each token of a weight's."""
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


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def make(cu, tokens, c, K, dtype, bias=True, state=True, seed=0):
    g = torch.Generator().manual_seed(900 + seed)
    n = len(cu) - 1
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"x": r(tokens, c).to(dtype), "w": r(c, K) * K ** -0.5, "b": 0.3 * r(c) if bias else None,
            "X0": r(n, K - 1, c).to(dtype) if state else None, "dy": r(tokens, c).to(dtype),
            "dX": r(n, K - 1, c).to(dtype) if state else None}


def dev(x):
    return {m: None if t is None else t.to(DEV) for m, t in x.items()}


def wide(t):
    return None if t is None else t.double()


def reference(cu, x, silu):
    leaves = {m: wide(x[m]) for m in ("x", "w", "b", "X0")}
    if leaves["X0"] is None:
        leaves["X0"] = torch.zeros((len(cu) - 1, x["w"].shape[1] - 1, x["x"].shape[1]), dtype=torch.float64)
    ins = {m: t.requires_grad_(True) for m, t in leaves.items() if t is not None}
    y, X, mag = R.conv(cu, *[ins.get(m) for m in ("x", "w", "b", "X0")], silu)
    dX = torch.zeros_like(X) if x["dX"] is None else wide(x["dX"])
    grads = dict(zip(ins, torch.autograd.grad((y, X), list(ins.values()), (wide(x["dy"]), dX), materialize_grads=True)))
    # sums of absolute terms of the gradients: |act'| <= 1.1
    a = {m: None if t is None else t.detach().abs() for m, t in ins.items()}
    p = {m: t.requires_grad_(True) for m, t in a.items() if t is not None}
    ya, Xa, _ = R.conv(cu, *[p.get(m) for m in ("x", "w", "b", "X0")], False)
    mags = dict(zip(p, torch.autograd.grad((ya, Xa), list(p.values()), (1.1 * wide(x["dy"]).abs(), dX.abs()),
                                           materialize_grads=True)))
    assert not mag.numel() or mag.max() <= 16
    return y, X, mag, grads, mags


def forward(cu, d, silu, X=None, y=None):
    y = torch.full_like(d["x"], 7.0) if y is None else y
    lq.leapquant_conv_forward(offsets(cu), d["x"], d["w"], y, bias=d["b"], activation="silu" if silu else "none",
                              X0=d["X0"], X=X)
    return y


def covered(cu, tokens):
    keep = torch.zeros(tokens, dtype=torch.bool)
    keep[cu[0]:cu[-1]] = True
    return keep


CASES = [([0, 1], 1, 1, 4), ([0, 5], 5, 64, 2), ([0, 0, 3, 3, 4, 40, 40], 40, 129, 4), ([2, 9, 70], 75, 512, 3),
         ([0, 31, 64, 66, 200], 200, 1000, 4), ([3, 3, 3], 6, 24, 4), ([0, 33, 34, 36, 39, 43, 160], 161, 8, 4),
         ([0, 2, 4, 5, 300], 300, 72, 4)]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("cu,tokens,c,K", CASES)
def test_conv_and_gradient(cu, tokens, c, K, dtype, silu):
    bias, state = tokens % 2 == 0, tokens != 300
    x = make(cu, tokens, c, K, dtype, bias, state, seed=tokens)
    d = dev(x)
    y_ref, X_ref, mag, grads, mags = reference(cu, x, silu)
    X = torch.full((len(cu) - 1, K - 1, c), 7.0, dtype=dtype, device=DEV)
    y = forward(cu, d, silu, X)
    keep = covered(cu, tokens)
    check(y[keep.to(DEV)], y_ref[keep], 16, "y", mag[keep])
    assert (y[~keep.to(DEV)] == 7).all()
    assert torch.equal(X.cpu().double(), X_ref.detach())
    out = {"x": torch.full_like(d["x"], 7.0), "w": torch.full_like(d["w"], 7.0), "b": torch.full((c,), 7.0, device=DEV),
           "X0": torch.full_like(X, 7.0)}
    ws = lq.leapquant_conv_workspace(tokens, len(cu) - 1, c, K)
    lq.leapquant_conv_backward(offsets(cu), d["x"], d["w"], d["dy"], out["x"], bias=d["b"],
                               activation="silu" if silu else "none", X0=d["X0"], dweight=out["w"],
                               dbias=out["b"] if bias else None, dX=d["dX"], dX0=out["X0"], workspace=ws)
    check(out["x"][keep.to(DEV)], grads["x"][keep], 64, "dx", mags["x"][keep])
    assert (out["x"][~keep.to(DEV)] == 7).all()
    check(out["w"], grads["w"], 64 + tokens, "dw", mags["w"])
    check(out["X0"], grads["X0"], 64, "dX0", mags["X0"])
    if bias:
        check(out["b"], grads["b"], 64 + tokens, "dbias", mags["b"])
    # without the optional gradients, the same dx
    again = torch.full_like(d["x"], 7.0)
    lq.leapquant_conv_backward(offsets(cu), d["x"], d["w"], d["dy"], again, bias=d["b"],
                               activation="silu" if silu else "none", X0=d["X0"], dX=d["dX"])
    assert torch.equal(again, out["x"])


@pytest.mark.parametrize("tokens", [8192, 33000])
def test_many_tokens(tokens):
    """Runs of 32 tokens and of more, one sequence much longer than the others."""
    cu, c, K = [0, 1, 3, 3, tokens - 40, tokens], 8, 4
    x = make(cu, tokens, c, K, F32, seed=3)
    d = dev(x)
    leaves = {m: d[m].double().requires_grad_(True) for m in ("x", "w", "b", "X0")}
    parts = []
    for i in range(len(cu) - 1):
        row = torch.cat((leaves["X0"][i], leaves["x"][cu[i]:cu[i + 1]]))
        n = cu[i + 1] - cu[i]
        parts.append(sum(row[j:j + n] * leaves["w"][:, j] for j in range(K)) + leaves["b"])
    v = torch.cat(parts)
    y_ref = v * torch.sigmoid(v)
    grads = torch.autograd.grad(y_ref, list(leaves.values()), d["dy"].double())
    check(forward(cu, d, True), y_ref, 16, "y", torch.tensor(16.0))
    out = {m: torch.empty_like(d[m]) for m in ("x", "w", "b", "X0")}
    lq.leapquant_conv_backward(offsets(cu), d["x"], d["w"], d["dy"], out["x"], bias=d["b"], X0=d["X0"], dweight=out["w"],
                               dbias=out["b"], dX0=out["X0"], workspace=lq.leapquant_conv_workspace(40000, 5, c, K))
    # |dy| <= 5, |x| <= 6, |act'| <= 1.1: a weight's terms sum to at most tokens * 33
    for m, g in zip(leaves, grads):
        many = m in ("w", "b")
        check(out[m], g, 64 + (tokens if many else 0), m, torch.tensor(33.0 * (tokens if many else 1)))


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,c,K", [(1, 1, 4), (5, 64, 2), (37, 513, 3), (64, 2048, 4)])
def test_step(rows, c, K, dtype, silu):
    """Slots in any order, some rows idle, the other slots left as they are; in place and not."""
    g = torch.Generator().manual_seed(rows)
    n = rows + 3
    x = make([0, rows], rows, c, K, dtype, rows % 2 == 0, seed=7)
    X = torch.randn((n, K - 1, c), generator=g).to(dtype)
    slots = torch.randperm(n, generator=g)[:rows].to(torch.int32)
    idle = torch.zeros(rows, dtype=torch.bool)
    if rows > 4:
        slots[1], slots[3] = -1, n
        idle[1] = idle[3] = True
    y_ref, X_ref = torch.full((rows, c), 7.0).double(), X.double()
    mag = torch.ones(1).double()
    for r in range(rows):
        if not idle[r]:
            s = int(slots[r])
            y_ref[r:r + 1], X_ref[s:s + 1], m = R.conv([0, 1], wide(x["x"][r:r + 1]), wide(x["w"]), wide(x["b"]),
                                                       wide(X[s:s + 1]), silu)
            mag = torch.maximum(mag, m.max())
    d = dev(x)
    kw = dict(bias=d["b"], activation="silu" if silu else "none", slots=slots.to(DEV))
    y, Xd, out = torch.full_like(d["x"], 7.0), X.to(DEV), torch.full_like(X, 7.0).to(DEV)
    lq.leapquant_conv_step(d["x"], d["w"], y, Xd, X_out=out, **kw)
    check(y, y_ref, 16, "y", mag)
    assert torch.equal(Xd.cpu(), X)
    listed = slots[~idle].long()
    assert torch.equal(out.cpu()[listed].double(), X_ref[listed])
    rest = torch.ones(n, dtype=torch.bool)
    rest[listed] = False
    assert (out.cpu()[rest] == 7).all()
    y2 = torch.full_like(y, 7.0)
    lq.leapquant_conv_step(d["x"], d["w"], y2, Xd, **kw)
    assert torch.equal(y, y2) and torch.equal(Xd.cpu().double(), X_ref)


def test_tokens_one_by_one_are_the_sequence():
    """A prompt, then its next tokens by steps: the same as the whole sequence, bit for bit."""
    cu, c, K = [0, 20, 21, 60], 256, 4
    x = make(cu, 60, c, K, BF16, seed=8)
    d = dev(x)
    X = torch.empty((3, K - 1, c), dtype=BF16, device=DEV)
    whole = forward(cu, d, True, X)
    for i in range(3):
        first = (cu[i + 1] - cu[i]) // 2
        part = {**d, "x": d["x"][cu[i]:cu[i] + first], "X0": d["X0"][i:i + 1]}
        Xi = torch.empty((1, K - 1, c), dtype=BF16, device=DEV)
        assert torch.equal(forward([0, first], part, True, Xi), whole[cu[i]:cu[i] + first])
        for t in range(cu[i] + first, cu[i + 1]):
            y = torch.empty((1, c), dtype=BF16, device=DEV)
            lq.leapquant_conv_step(d["x"][t:t + 1], d["w"], y, Xi, bias=d["b"])
            assert torch.equal(y, whole[t:t + 1])
        assert torch.equal(Xi[0], X[i])


@pytest.mark.parametrize("c,pad,off", [(64, 8, 0), (64, 8, 3), (65, 6, 1), (64, 5, 8)])
def test_strided_rows(c, pad, off):
    """Slices of a wider row, aligned to 16 bytes and not: the same results."""
    cu = [0, 12, 40]
    x = make(cu, 40, c, 4, BF16, seed=9)
    d = dev(x)
    ref = forward(cu, d, True)
    big = torch.full((40, c + pad + off), 7.0, dtype=BF16, device=DEV)
    big[:, off:off + c] = d["x"]
    out = torch.full((40, c + pad + off), 9.0, dtype=BF16, device=DEV)
    forward(cu, {**d, "x": big[:, off:off + c]}, True, y=out[:, off:off + c])
    assert torch.equal(out[:, off:off + c], ref) and (out[:, :off] == 9).all() and (out[:, off + c:] == 9).all()
    dx = torch.empty_like(d["x"])
    lq.leapquant_conv_backward(offsets(cu), d["x"], d["w"], d["dy"], dx, bias=d["b"], X0=d["X0"], dX=d["dX"])
    out.fill_(9.0)
    lq.leapquant_conv_backward(offsets(cu), big[:, off:off + c], d["w"], d["dy"], out[:, off:off + c], bias=d["b"],
                               X0=d["X0"], dX=d["dX"])
    # (sums in another order of channels per lane: the same terms, bit for bit)
    assert torch.equal(out[:, off:off + c], dx) and (out[:, off + c:] == 9).all()


def test_one_row_for_all_tokens():
    """An input of token stride 0."""
    d = dev(make([0, 50], 50, 128, 4, F16, state=False, seed=10))
    row = d["x"][:1].expand(50, 128)
    assert torch.equal(forward([0, 50], {**d, "x": row}, True, y=torch.empty_like(d["x"])),
                       forward([0, 50], {**d, "x": row.contiguous()}, True))


def test_far_offsets():
    """Element offsets beyond 2^31."""
    T, c, stride = 600, 64, 4_000_000
    d = dev(make([0, T], T, c, 4, BF16, state=False, seed=11))
    far = torch.empty(T * stride, dtype=BF16, device=DEV).as_strided((T, c), (stride, 1))
    far.copy_(d["x"])
    out = torch.empty(T * stride, dtype=BF16, device=DEV).as_strided((T, c), (stride, 1))
    assert torch.equal(forward([0, T], {**d, "x": far}, True, y=out), forward([0, T], d, True))


def test_values_that_are_not_finite_stay_where_the_formula_has_them():
    cu = [0, 10, 20]
    x = make(cu, 20, 16, 4, F32, seed=12)
    clean = forward(cu, dev(x), True)
    x["x"][7, 3] = float("nan")
    x["x"][8, 5] = float("inf")
    y = forward(cu, dev(x), True).cpu()
    hit = torch.zeros(20, 16, dtype=torch.bool)
    hit[7:10, 3] = True
    hit[8:10, 5] = True
    assert torch.equal(y[~hit], clean.cpu()[~hit]) and y[7:10, 3].isnan().all()


def test_offsets_that_do_not_ascend_stay_in_bounds():
    """Unspecified results, but no access outside the arrays (offsets are held to [0, tokens])."""
    d = dev(make([0, 8, 16, 24], 24, 64, 4, F32, seed=13))
    for cu in ([9, 3, 24, 0], [-5, 1 << 30, 7, 1 << 30], [24, 24, 24, 24], [30, 40, 50, 60]):
        guard = torch.full((3, 24, 64), 7.0, device=DEV)
        forward(cu, d, True, torch.empty_like(d["X0"]), y=guard[1])
        assert (guard[0] == 7).all() and (guard[2] == 7).all()
        ws = lq.leapquant_conv_workspace(24, 3, 64, 4)
        lq.leapquant_conv_backward(offsets(cu), d["x"], d["w"], d["dy"], guard[1], bias=d["b"], X0=d["X0"],
                                   dweight=torch.empty_like(d["w"]), dX=d["dX"], dX0=torch.empty_like(d["X0"]), workspace=ws)
        assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_no_tokens():
    d = dev(make([0, 0, 0], 0, 32, 4, F32, seed=14))
    X = torch.empty_like(d["X0"])
    forward([0, 0, 0], d, True, X)
    assert torch.equal(X, d["X0"])
    dw, dX0 = torch.full_like(d["w"], 7.0), torch.empty_like(d["X0"])
    lq.leapquant_conv_backward(offsets([0, 0, 0]), d["x"], d["w"], d["dy"], torch.empty_like(d["x"]), X0=d["X0"], dweight=dw,
                               dX=d["dX"], dX0=dX0)
    assert (dw == 0).all() and torch.equal(dX0, d["dX"])


def test_captured_step_on_another_stream():
    """A captured step, replayed with the program's own work between, is the eager steps."""
    g = torch.Generator().manual_seed(15)
    d = dev(make([0, 9], 9, 320, 4, BF16, seed=15))
    X = torch.randn((9, 3, 320), generator=g).to(DEV, BF16)
    eager, x, y = X.clone(), d["x"].clone(), torch.empty_like(d["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lq.leapquant_conv_step(x, d["w"], y, X.clone(), bias=d["b"])  # warm-up
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lq.leapquant_conv_step(x, d["w"], y, X, bias=d["b"])
    torch.cuda.synchronize()
    for k in range(4):
        x.copy_((d["x"] * (k + 1)).to(BF16))
        graph.replay()
        y2 = torch.empty_like(y)
        lq.leapquant_conv_step(x, d["w"], y2, eager, bias=d["b"])
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(X, eager)


def test_refusals_on_the_device():
    d = dev(make([0, 4, 10], 10, 32, 4, F32, seed=16))
    ok = dict(cu_seqlens=offsets([0, 4, 10]), x=d["x"], weight=d["w"], y=torch.empty_like(d["x"]))
    lq.leapquant_conv_forward(**ok)
    bad = [dict(cu_seqlens=ok["cu_seqlens"].long()), dict(cu_seqlens=ok["cu_seqlens"].cpu()), dict(weight=d["w"].half()),
           dict(weight=d["w"][:16]), dict(y=torch.empty(10, 31, device=DEV)), dict(y=ok["y"].cpu()), dict(y=ok["y"].half()),
           dict(x=d["x"].t().contiguous().t()), dict(bias=torch.zeros(31, device=DEV)), dict(X0=d["X0"][:1]),
           dict(X0=d["X0"].half()), dict(activation="sigmoid")]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            lq.leapquant_conv_forward(**{**ok, **kw})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_conv_forward(**{**ok, "y": d["x"]})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_conv_forward(**ok, X0=d["X0"], X=d["X0"])
    with pytest.raises(lq.LeapQuantError):   # a weight gradient without a workspace
        lq.leapquant_conv_backward(ok["cu_seqlens"], d["x"], d["w"], d["dy"], ok["y"], dweight=torch.empty_like(d["w"]))
