"""Forms of the calls around the recurrence that the larger tests leave out:
thousands of sequences, most of them empty; inputs shared by tokens or groups; a
training step of the convolution and the norm in a captured graph."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import scan_beside
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


def scan_inputs(T, c, N, G, n, seed, dtype=F32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    low = lambda *s: r(*s).to(dtype)  # noqa: E731
    return {"x": low(T, c), "dt": low(T, c) - 2, "A": -torch.exp(r(c, N)), "B": low(T, G, N), "C": low(T, G, N), "D": r(c),
            "bias": r(c), "z": low(T, c), "S0": r(n, c, N), "dy": low(T, c), "dS": r(n, c, N)}


def scan_both(where, d, out, dS0, softplus=True):
    """Forward and backward into `out`; returns y and S."""
    (T, c), (_, N) = d["x"].shape, d["A"].shape
    plan = lq.LeapQuantScan(T, where.numel() - 1, c, N, groups=d["B"].shape[1], dtype=d["x"].dtype, softplus=softplus, save=True)
    plan.workspace.fill_(255)
    y, S = torch.full(d["x"].shape, 7.0, dtype=d["x"].dtype, device=DEV), torch.full_like(dS0, 7.0)
    kw = dict(D=d["D"], dt_bias=d["bias"], z=d["z"])
    lq.leapquant_scan_forward(plan, where, d["x"], d["dt"], d["A"], d["B"], d["C"], y, S0=d["S0"], S=S, **kw)
    lq.leapquant_scan_backward(plan, where, d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], out["x"], out["dt"], out["A"],
                               out["B"], out["C"], dD=out.get("D"), ddt_bias=out.get("bias"), dz=out.get("z"), dS=d["dS"],
                               dS0=dS0, **kw)
    return y, S


def test_thousands_of_sequences_most_of_them_empty():
    """4,001 sequences of 600 tokens: two of many tokens, a hundred of one, the others of none, at both ends too."""
    g = torch.Generator().manual_seed(1)
    lens = torch.zeros(4001, dtype=torch.long)
    lens[torch.randperm(3990, generator=g)[:100] + 5] = 1
    for i, m in ((1500, 199), (3991, 601 - 200 - int(lens.sum()) + int(lens[1500]))):
        lens[i] = m
    cu = [0, *lens.cumsum(0).tolist()]
    T, n, c, N = cu[-1], len(lens), 24, 8
    where = torch.tensor(cu, dtype=torch.int32, device=DEV)
    d = scan_inputs(T, c, N, 1, n, 2)
    out = {m: torch.full_like(d[m], 7.0) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z")}
    dS0 = torch.full_like(d["S0"], 7.0)
    y, S = scan_both(where, d, out, dS0)
    args = [d[m].double() for m in ("x", "dt", "A", "B", "C", "D", "bias", "z", "S0", "dy", "dS")]
    ref, top = (scan_beside.scan_adjoint(cu, *args, absolute=a) for a in (False, True))
    most = int(lens.max())
    k = 9 * most + 2 * N + c + 160
    check(y, ref["y"], 4 * most + N + 64, "y", top["y"])
    check(S, ref["S"], 4 * most + 32, "S", top["S"])
    check(dS0, ref["S0"], k, "dS0", top["S0"])
    for m, t in out.items():
        check(t, ref[m], k + T, "d" + m, top[m])
    empty = (lens == 0).to(DEV)
    assert torch.equal(S[empty], d["S0"][empty]) and torch.equal(dS0[empty], d["dS"][empty])
    # the convolution: the same sequences one call each are the whole, bit for bit
    w, X0 = 0.5 * d["A"][:, :4].contiguous(), d["S0"][:, :, :3].transpose(1, 2).contiguous()
    dX = d["dS"][:, :, :3].transpose(1, 2).contiguous()
    y, X, dx, dX0 = torch.full_like(d["x"], 7.0), torch.full_like(X0, 7.0), torch.full_like(d["x"], 7.0), torch.full_like(X0, 7.0)
    lq.leapquant_conv_forward(where, d["x"], w, y, X0=X0, X=X)
    lq.leapquant_conv_backward(where, d["x"], w, d["dy"], dx, X0=X0, dX=dX, dX0=dX0)
    assert torch.equal(X[empty], X0[empty]) and torch.equal(dX0[empty], dX[empty])
    for i in torch.nonzero(lens).flatten().tolist():
        at, one = slice(cu[i], cu[i + 1]), torch.tensor([0, cu[i + 1] - cu[i]], dtype=torch.int32, device=DEV)
        y1, dx1 = torch.empty_like(d["x"][at]), torch.empty_like(d["x"][at])
        X1, dX1 = torch.empty_like(X0[:1]), torch.empty_like(X0[:1])
        lq.leapquant_conv_forward(one, d["x"][at], w, y1, X0=X0[i:i + 1], X=X1)
        lq.leapquant_conv_backward(one, d["x"][at], w, d["dy"][at], dx1, X0=X0[i:i + 1], dX=dX[i:i + 1], dX0=dX1)
        assert torch.equal(y1, y[at]) and torch.equal(X1[0], X[i]) and torch.equal(dx1, dx[at]) and torch.equal(dX1[0], dX0[i])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_inputs_that_tokens_or_groups_share(dtype):
    """A row for all tokens, a B and C for all groups (strides of zero): as copies of them."""
    T, c, N, G, cu = 300, 96, 16, 3, [0, 90, 300]
    where = torch.tensor(cu, dtype=torch.int32, device=DEV)
    d = scan_inputs(T, c, N, G, 2, 3, dtype)
    shared = {**d, "dt": d["dt"][:1].expand(T, c), "z": d["z"][5:6].expand(T, c), "dy": d["dy"][:1].expand(T, c),
              "B": d["B"][:, :1].expand(T, G, N), "C": d["C"][:1].expand(T, G, N)}
    runs = []
    for v in (shared, {m: t.contiguous() for m, t in shared.items()}):
        out = {m: torch.full(d[m].shape, 7.0, dtype=d[m].dtype, device=DEV) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z")}
        dS0 = torch.full_like(d["S0"], 7.0)
        runs.append((*scan_both(where, v, out, dS0), dS0, *out.values()))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    # the norm: one gate for all heads, one residual row for all tokens
    a = d["x"].view(T, 3, 32)
    z, res = d["z"][:, :32].unsqueeze(1).expand(T, 3, 32), d["S0"][0, :, 0].contiguous().view(1, 3, 32).expand(T, 3, 32)
    got = []
    for f in (lambda t: t, torch.Tensor.contiguous):
        h, y = torch.full((T, 3, 32), 7.0, device=DEV), torch.full((T, 3, 32), 7.0, dtype=dtype, device=DEV)
        lq.leapquant_block_norm(a, h=h, y=y, z=f(z), res=f(res), out_norm=True)
        da, dz, dres = torch.empty_like(y), torch.empty_like(y), torch.empty_like(h)
        lq.leapquant_block_norm_backward(a, da, dh=f(res), dy=f(z), z=f(z), res=f(res), out_norm=True, dz=dz, dres=dres)
        got.append((h, y, da, dz, dres))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_captured_training_step_of_convolution_and_norm():
    """Both with their weights' gradients, whose sums take a second launch, in one graph, replayed with the program's own
    work between."""
    cu, T, c, K = [0, 700, 9000, 9500], 9500, 512, 4
    where = torch.tensor(cu, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    first = r(T, c).to(BF16)
    d = {"x": first.clone(), "w": r(c, K), "b": r(c), "X0": r(3, K - 1, c).to(BF16), "dh": r(T, 1, c), "dy": r(T, 1, c).to(BF16),
         "res": r(T, 1, c), "wi": r(c), "wo": r(c), "dX": r(3, K - 1, c).to(BF16)}

    def buffers():
        e = torch.empty_like
        return {"u": e(first), "X": e(d["X0"]), "h": e(d["dh"]), "y": e(d["dy"]), "du": e(first), "dx": e(first), "dw": e(d["w"]),
                "db": e(d["b"]), "dX0": e(d["X0"]), "dres": e(d["dh"]), "dwi": e(d["wi"]), "dwo": e(d["wo"]),
                "one": lq.leapquant_conv_workspace(T, 3, c, K).fill_(255),
                "two": lq.leapquant_block_norm_workspace(T, 1, c).fill_(255)}

    def step(o):
        lq.leapquant_conv_forward(where, d["x"], d["w"], o["u"], bias=d["b"], X0=d["X0"], X=o["X"])
        kw = dict(res=d["res"], scale=0.5, out_norm=True, out_weight=d["wo"], in_weight=d["wi"])
        lq.leapquant_block_norm(o["u"][:, None], h=o["h"], y=o["y"], **kw)
        lq.leapquant_block_norm_backward(o["u"][:, None], o["du"][:, None], dh=d["dh"], dy=d["dy"], dres=o["dres"],
                                         dout_weight=o["dwo"], din_weight=o["dwi"], workspace=o["two"], **kw)
        lq.leapquant_conv_backward(where, d["x"], d["w"], o["du"], o["dx"], bias=d["b"], X0=d["X0"], dweight=o["dw"],
                                   dbias=o["db"], dX=d["dX"], dX0=o["dX0"], workspace=o["one"])

    o = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(o)
    torch.cuda.synchronize()
    for k in range(4):
        d["x"].copy_((first.float() * (1 + 0.5 * k)).to(BF16))
        graph.replay()
        eager = buffers()
        step(eager)
        torch.cuda.synchronize()
        for m in o:
            if m not in ("one", "two"):
                assert torch.equal(o[m], eager[m]), (k, m)
