"""Norm of query and key heads with the position rotation on the GPU, against
its 64-bit form.

Bounds (R.bound): a forward value stands behind a sum of 128 squares, a square
root and a quotient, the weight, the scale, and the rotation's two products,
whose sine and cosine are off by up to 2^-23 (a fraction of a turn rounded to
32 bits): n = 160 roundings of 2^-24.  A gradient stands behind twice that."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import sequence_reference as R

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


def make(T, hq, hk, dtype, weight, rot, seed=0, far=1 << 17):
    g = torch.Generator().manual_seed(500 + seed)
    x = {"q": (3 * torch.randn((T, hq, 128), generator=g)).to(dtype),
         "k": (3 * torch.randn((T, hk, 128), generator=g)).to(dtype)}
    x["wq"], x["wk"] = ((1 + 0.2 * torch.randn(128, generator=g)) if weight else None for _ in range(2))
    x["pos"] = torch.randint(0, far, (T,), generator=g) if rot else None
    x["freq"] = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2)) if rot else None
    x["gq"], x["gk"] = torch.randn((T, hq, 128), generator=g), torch.randn((T, hk, 128), generator=g)
    return x


def how(x, kind, scale, interleaved):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return dict(norm=kind, eps=1e-5, q_weight=d(x["wq"]), k_weight=d(x["wk"]), q_scale=scale, positions=d(x["pos"]),
                inv_freq=d(x["freq"]), interleaved=interleaved)


def reference(x, kind, scale, interleaved, out):
    names = [m for m in ("q", "k", "wq", "wk") if x[m] is not None]
    leaf = {m: x[m].double().requires_grad_(True) for m in names}
    y = {m: R.head_norm(leaf[m], kind, 1e-5, leaf.get("w" + m), s, x["pos"], x["freq"], interleaved)
         for m, s in (("q", scale), ("k", 1.0))}
    loss = sum((y[m] * x["g" + m].to(out).double()).sum() for m in ("q", "k"))
    return y, dict(zip(names, torch.autograd.grad(loss, [leaf[m] for m in names])))


CASES = [(1, 1, 1, "l2", False, 0, False), (3, 4, 2, "rms", True, 128, True), (5, 2, 5, "l2", True, 64, False),
         (67, 17, 3, "rms", False, 96, False), (130, 16, 16, "l2", False, 16, True), (9, 33, 1, "rms", True, 32, True),
         (2, 3, 0, "l2", False, 128, False), (700, 2, 1, "rms", True, 128, False)]


@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,hq,hk,kind,weight,rot,interleaved", CASES)
def test_norm_and_gradient(T, hq, hk, kind, weight, rot, interleaved, dtype, out):
    x = make(T, hq, hk, dtype, weight, rot, seed=T)
    args = how(x, kind, 0.37, interleaved)
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    y = {"q": torch.empty((T, hq, 128), dtype=out, device=DEV), "k": torch.empty((T, hk, 128), dtype=out, device=DEV)}
    lq.leapquant_head_norm(q, k, y["q"], y["k"], **args)
    ref, grads = reference(x, kind, 0.37, interleaved, out)
    for m in ("q", "k"):
        R.check(y[m], ref[m], 160, m)
    d = {"q": torch.empty_like(q), "k": torch.empty_like(k)}
    for m in ("wq", "wk"):
        d[m] = torch.full((128,), 7.0, device=DEV) if weight else None
    ws = lq.leapquant_head_norm_workspace(T, hq, hk)
    lq.leapquant_head_norm_backward(q, k, x["gq"].to(DEV, out), x["gk"].to(DEV, out), d["q"], d["k"],
                                    dq_weight=d["wq"], dk_weight=d["wk"], workspace=ws if weight else None, **args)
    for m, r in grads.items():
        # a weight's gradient sums a term for every token and head, each about as large as the others
        R.check(d[m], r, 320 + (T * max(hq, hk) if m[0] == "w" else 0), "d" + m)


def test_far_positions():
    """Positions up to 2^40: the angle's product and reduction keep 64 bits (2^-53 of 2^40 radians: 2^-13)."""
    x = make(50, 2, 2, F32, False, 64, seed=1, far=1 << 40)
    x["freq"] = x["freq"] * 2.0 ** -20  # angles up to 2^20: 2^-33 of a radian after the product
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    lq.leapquant_head_norm(q, k, yq, yk, **how(x, "l2", 1.0, False))
    ref, _ = reference(x, "l2", 1.0, False, F32)
    R.check(yq, ref["q"], 160, "q")
    R.check(yk, ref["k"], 160, "k")


@pytest.mark.parametrize("kind", ["l2", "rms"])
def test_zero_heads(kind):
    x = make(4, 2, 1, F32, True, 32, seed=2)
    x["q"][1] = 0.0
    x["k"][2, 0] = 0.0
    args = how(x, kind, 1.0, False)
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    yq, yk, dq, dk = (torch.empty_like(t) for t in (q, k, q, k))
    lq.leapquant_head_norm(q, k, yq, yk, **args)
    lq.leapquant_head_norm_backward(q, k, x["gq"].to(DEV), x["gk"].to(DEV), dq, dk, **args)
    ref, grads = reference(x, kind, 1.0, False, F32)
    assert (yq[1] == 0).all() and (yk[2, 0] == 0).all()
    R.check(yq, ref["q"], 160, "q")
    R.check(dq, grads["q"], 320, "dq")
    R.check(dk, grads["k"], 320, "dk")


def test_strided_in_place_and_empty():
    x = make(21, 3, 2, BF16, True, 128, seed=3)
    args = how(x, "rms", 0.5, False)
    ref, _ = reference(x, "rms", 0.5, False, BF16)
    rows = torch.full((21, 7, 128), 7.0, dtype=BF16, device=DEV)
    q, k = rows[:, 1:4], rows[:, 4:6]
    q.copy_(x["q"])
    k.copy_(x["k"])
    lq.leapquant_head_norm(q, k, q, k, **args)
    R.check(q, ref["q"], 160, "q")
    R.check(k, ref["k"], 160, "k")
    assert (rows[:, 0] == 7).all() and (rows[:, 6] == 7).all()
    # no tokens: nothing to do, weight gradients of zero
    none = torch.empty((0, 3, 128), dtype=BF16, device=DEV)
    dw = torch.full((128,), 7.0, device=DEV)
    args["positions"] = args["positions"][:0]
    lq.leapquant_head_norm(none, none[:, :2], none.clone(), none[:, :2].clone(), **args)
    lq.leapquant_head_norm_backward(none, none[:, :2], none.clone(), none[:, :2].clone(), none.clone(),
                                    none[:, :2].clone(), dq_weight=dw, workspace=lq.leapquant_head_norm_workspace(0, 3, 2),
                                    **args)
    assert (dw == 0).all()


def test_large_and_repeatable():
    """More heads than one pass of the backward's workgroups holds; the weights' sums do not depend on timing."""
    T, hq, hk = 3001, 20, 13
    g = torch.Generator(device=DEV).manual_seed(9)
    q, k = (torch.randn((T, h, 128), generator=g, device=DEV).to(BF16) for h in (hq, hk))
    gq, gk = (torch.randn((T, h, 128), generator=g, device=DEV) for h in (hq, hk))
    w = 1 + 0.1 * torch.randn(128, generator=g, device=DEV)
    pos = torch.arange(T, device=DEV)
    freq = 10000.0 ** (-torch.arange(48, dtype=torch.float64, device=DEV) / 48)
    args = dict(norm="rms", q_weight=w, k_weight=w, positions=pos, inv_freq=freq)
    runs = []
    for _ in range(2):
        dq, dk, dwq, dwk = torch.empty_like(q), torch.empty_like(k), torch.empty_like(w), torch.empty_like(w)
        lq.leapquant_head_norm_backward(q, k, gq, gk, dq, dk, dq_weight=dwq, dk_weight=dwk,
                                        workspace=lq.leapquant_head_norm_workspace(T, hq, hk), **args)
        runs.append((dq, dk, dwq, dwk))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    leaves = [t.double().requires_grad_(True) for t in (q, k, w, w)]
    y = [R.head_norm(leaves[i], "rms", 1e-6, leaves[2 + i], 1.0, pos, freq, False) for i in range(2)]
    ref = torch.autograd.grad((y[0] * gq).sum() + (y[1] * gk).sum(), leaves)
    for got, want, n, name in zip(runs[0], ref, (320, 320, 320 + T * hq, 320 + T * hk), ("dq", "dk", "dwq", "dwk")):
        R.check(got, want, n, name)


def test_captured():
    x = make(40, 4, 4, BF16, True, 64, seed=4)
    args = how(x, "l2", 1.0, True)
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    yq, yk, dq, dk = (torch.empty_like(t) for t in (q, k, q, k))
    dw = torch.empty(128, device=DEV)
    ws = lq.leapquant_head_norm_workspace(40, 4, 4)

    def step():
        lq.leapquant_head_norm(q, k, yq, yk, **args)
        lq.leapquant_head_norm_backward(q, k, yk, yq, dq, dk, dq_weight=dw, workspace=ws, **args)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for i in range(4):
        q.copy_(torch.randn(q.shape, device=DEV))
        step()
        want = [t.clone() for t in (yq, yk, dq, dk, dw)]
        for t in (yq, yk, dq, dk, dw):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((yq, yk, dq, dk, dw), want):
            assert torch.equal(a, b)


def test_keys_alone_and_the_gradient_of_unit_weights():
    T, hk = 37, 21
    x = make(T, 0, hk, BF16, False, 64, seed=6)
    args = how(x, "rms", 1.0, False)
    q, k = x["q"].to(DEV), x["k"].to(DEV)
    y, dk, dw = torch.empty((T, hk, 128), device=DEV), torch.empty_like(k), torch.empty(128, device=DEV)
    lq.leapquant_head_norm(q, k, q.float(), y, **args)
    lq.leapquant_head_norm_backward(q, k, q.float(), x["gk"].to(DEV), torch.empty_like(q), dk, dk_weight=dw,
                                    workspace=lq.leapquant_head_norm_workspace(T, 0, hk), **args)
    leaves = [x["k"].double().requires_grad_(True), torch.ones(128, dtype=torch.float64, requires_grad=True)]
    ref = R.head_norm(leaves[0], "rms", 1e-5, leaves[1], 1.0, x["pos"], x["freq"], False)
    R.check(y, ref, 160, "k")
    for got, want, n, name in zip((dk, dw), torch.autograd.grad((ref * x["gk"].double()).sum(), leaves),
                                  (320, 320 + T * hk), ("dk", "dw")):
        R.check(got, want, n, name)
