"""The operators around the recurrence together, as a layer uses them.

Bounds: an operator's own roundings (layer_reference, sequence_reference) and
those that it is handed.  The delta rule takes queries, keys and values that are
176 roundings off (convolution 16, head norm 160); an error of a key enters each
later token's update twice, so n = 2 T * 176 + 256 + 3 T for its outputs, and the
norm of a head passes an error of its input on at most twice (its own value and
the root): n = 2 (355 T + 256) + 320.  The scan takes values 16 roundings off and
is linear in them: n = 16 + 4 T + N + 64, and the norm of the stream doubles it.
Gradients through all three: each operator's n twice, 9 T + 4 dim + 2 N + per +
400, once more for each later one: n = 4 (9 T + 4 dim + 2 N + per + 400)."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import layer_reference as R
from tests import sequence_reference as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def test_a_delta_rule_layer():
    """Convolution of queries, keys and values, head norm, recurrence, gated norm of its heads: prompts of three
    sequences, then each one's next tokens by a call of one token a sequence, against the 64-bit forms in a row."""
    cu, hk, hv, more = [0, 20, 21, 90], 2, 4, 3
    lens = [b - a + more for a, b in zip(cu, cu[1:])]
    c = (2 * hk + hv) * 128
    g = torch.Generator().manual_seed(60)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    full = [sum(lens[:i]) for i in range(4)]
    T = full[-1]
    x, w, z = r(T, c), r(c, 4) * 0.5, r(T, hv, 128)
    beta, alpha, wo = torch.sigmoid(r(T, hv)), torch.exp(-0.1 * torch.rand((T, hv), generator=g)), 1 + 0.1 * r(128)
    # 64 bits, whole sequences
    v64 = R.conv(full, x.double(), w.double(), None, torch.zeros((3, 3, c)).double(), True)[0].unflatten(1, (-1, 128))
    q64, k64 = (Q.head_norm(t, "l2", 1e-6, None, s, None, None, False) for t, s in
                ((v64[:, :hk], 128 ** -0.5), (v64[:, hk:2 * hk], 1.0)))
    o64, S64 = Q.recurrence(full, q64, k64, v64[:, 2 * hk:], beta.double(), alpha.double(),
                            torch.zeros((3 * hv, 128, 128)).double())
    h64, _ = R.block_norm(o64, z.double(), None, "silu", 1.0, True, wo.double(), None, 1e-6)
    # the kernels, prompts first
    d = [t.to(DEV) for t in (x, w, z, beta, alpha, wo)]
    X, S = torch.empty((3, 3, c), device=DEV), torch.empty((3 * hv, 128, 128), device=DEV)
    plan = lq.LeapQuantSequence(T, 3, hk, hv, dtype=F32)

    def layer(rows, where, S0, convolved):
        y = convolved.unflatten(1, (-1, 128))
        q, k = torch.empty((len(rows), hk, 128), device=DEV), torch.empty((len(rows), hk, 128), device=DEV)
        lq.leapquant_head_norm(y[:, :hk], y[:, hk:2 * hk], q, k, q_scale=128 ** -0.5)
        o, h = (torch.empty((len(rows), hv, 128), device=DEV) for _ in range(2))
        lq.leapquant_sequence_forward(plan, where, q, k, y[:, 2 * hk:], d[3][rows], d[4][rows], o, S0=S0, S=S)
        lq.leapquant_block_norm(o, h=h, z=d[2][rows], out_norm=True, out_weight=d[5])
        return h

    rows = torch.cat([torch.arange(full[i], full[i + 1] - more) for i in range(3)])
    y = torch.empty((len(rows), c), device=DEV)
    lq.leapquant_conv_forward(offsets(cu), d[0][rows], d[1], y, X=X)
    n = 2 * (355 * max(lens) + 256) + 320
    Q.check(layer(rows, offsets(cu), None, y), h64[rows], n, "prompts")
    for t in range(more):
        rows = torch.tensor([full[i + 1] - more + t for i in range(3)])
        y = torch.empty((3, c), device=DEV)
        lq.leapquant_conv_step(d[0][rows], d[1], y, X)
        Q.check(layer(rows, offsets([0, 1, 2, 3]), S, y), h64[rows], n, f"token {t}")
    Q.check(S, S64, n, "S")


def ssm_weights(g, c, dim, N):
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"w": r(c, 4) * 0.5, "b": 0.1 * r(c), "A": -torch.rand((c, N), generator=g) * 4 - 0.1, "D": r(c), "bias": r(c) - 2,
            "wi": 1 + 0.1 * r(dim)}


def test_a_state_space_layer_prompts_and_tokens():
    """Convolution, scan and the join to the stream, prompts and then tokens of some of the slots, one graph a token."""
    cu, c, N, more = [0, 40, 41, 130], 64, 16, 4
    lens = [b - a + more for a, b in zip(cu, cu[1:])]
    full = [sum(lens[:i]) for i in range(4)]
    T = full[-1]
    g = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, z, dt, B, C, res = r(T, c), r(T, c), r(T, c), r(T, 1, N), r(T, 1, N), r(T, 1, c)
    w = ssm_weights(g, c, c, N)
    e = {m: t.double() for m, t in w.items()}
    y64 = R.conv(full, x.double(), e["w"], e["b"], torch.zeros((3, 3, c)).double(), True)[0]
    s64, S64 = R.scan(full, y64, dt.double(), e["A"], B.double(), C.double(), e["D"], e["bias"], z.double(),
                      torch.zeros((3, c, N)).double())
    h64, n64 = R.block_norm(s64[:, None], None, res.double(), "none", 0.5, False, None, e["wi"], 1e-6)
    d = {m: t.to(DEV) for m, t in w.items()}
    x, z, dt, B, C, res = (t.to(DEV) for t in (x, z, dt, B, C, res))
    # slots of five running sequences; ours are 3, 0 and 4
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device=DEV)
    X, S = torch.full((5, 3, c), 7.0, device=DEV), torch.full((5, c, N), 7.0, device=DEV)
    rows = torch.cat([torch.arange(full[i], full[i + 1] - more) for i in range(3)]).to(DEV)
    y, s, Xp, Sp = (torch.empty(v, device=DEV) for v in ((len(rows), c), (len(rows), c), (3, 3, c), (3, c, N)))
    plan = lq.LeapQuantScan(len(rows), 3, c, N, dtype=F32)
    lq.leapquant_conv_forward(offsets(cu), x[rows], d["w"], y, bias=d["b"], X=Xp)
    lq.leapquant_scan_forward(plan, offsets(cu), y, dt[rows], d["A"], B[rows], C[rows], s, D=d["D"], dt_bias=d["bias"],
                              z=z[rows], S=Sp)
    h, out = (torch.empty((len(rows), 1, c), device=DEV) for _ in range(2))
    lq.leapquant_block_norm(s[:, None], h=h, y=out, res=res[rows], scale=0.5, in_weight=d["wi"])
    n = 2 * (16 + 4 * max(lens) + N + 64) + 2 * c + 64
    Q.check(h, h64[rows.cpu()], n, "h")
    Q.check(out, n64[rows.cpu()], n, "y")
    X[slots.long()], S[slots.long()] = Xp, Sp
    # a token of each sequence in one captured graph, a fourth row idle
    which = torch.tensor([3, 0, 4, -1], dtype=torch.int32, device=DEV)
    ins = {m: torch.zeros((4, *t.shape[1:]), device=DEV) for m, t in (("x", x), ("z", z), ("dt", dt), ("B", B), ("C", C),
                                                                     ("res", res))}
    y, s, h, out = (torch.zeros(v, device=DEV) for v in ((4, c), (4, c), (4, 1, c), (4, 1, c)))

    def token():
        lq.leapquant_conv_step(ins["x"], d["w"], y, X, bias=d["b"], slots=which)
        lq.leapquant_scan_step(y, ins["dt"], d["A"], ins["B"], ins["C"], s, S, D=d["D"], dt_bias=d["bias"], z=ins["z"],
                               slots=which)
        lq.leapquant_block_norm(s[:, None], h=h, y=out, res=ins["res"], scale=0.5, in_weight=d["wi"])

    keep = X.clone(), S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            token()
    torch.cuda.synchronize()
    X.copy_(keep[0])
    S.copy_(keep[1])
    for t in range(more):
        at = torch.tensor([full[i + 1] - more + t for i in range(3)])
        for m, v in (("x", x), ("z", z), ("dt", dt), ("B", B), ("C", C), ("res", res)):
            ins[m][:3] = v[at.to(DEV)]
        graph.replay()
        torch.cuda.synchronize()
        Q.check(h[:3], h64[at], n, f"h of token {t}")
        Q.check(out[:3], n64[at], n, f"y of token {t}")
    Q.check(S[slots.long()], S64, n, "S")
    assert (S[[1, 2]] == 7).all() and (X[[1, 2]] == 7).all()


def test_a_state_space_layer_in_training():
    """The three gradients one after another, in training's order, against automatic differentiation in 64 bits."""
    cu, c, N, T = [0, 30, 31, 100], 48, 8, 100
    g = torch.Generator().manual_seed(62)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    ins = {"x": r(T, c), "z": r(T, c), "dt": r(T, c), "B": r(T, 1, N), "C": r(T, 1, N), "res": r(T, 1, c), **ssm_weights(g, c, c, N)}
    dh, dy = r(T, 1, c), r(T, 1, c)
    e = {m: t.double().requires_grad_(True) for m, t in ins.items()}
    y64 = R.conv(cu, e["x"], e["w"], e["b"], torch.zeros((3, 3, c)).double(), True)[0]
    s64, _ = R.scan(cu, y64, e["dt"], e["A"], e["B"], e["C"], e["D"], e["bias"], e["z"], torch.zeros((3, c, N)).double())
    outs = R.block_norm(s64[:, None], None, e["res"], "none", 0.5, False, None, e["wi"], 1e-6)
    ref = dict(zip(e, torch.autograd.grad(outs, list(e.values()), (dh.double(), dy.double()))))
    d = {m: t.to(DEV) for m, t in ins.items()}
    new = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    where, plan = offsets(cu), lq.LeapQuantScan(T, 3, c, N, dtype=F32, save=True)
    y, s, h, o = new(T, c), new(T, c), new(T, 1, c), new(T, 1, c)
    lq.leapquant_conv_forward(where, d["x"], d["w"], y, bias=d["b"])
    more = dict(D=d["D"], dt_bias=d["bias"], z=d["z"])
    lq.leapquant_scan_forward(plan, where, y, d["dt"], d["A"], d["B"], d["C"], s, **more)
    join = dict(res=d["res"], scale=0.5, in_weight=d["wi"])
    lq.leapquant_block_norm(s[:, None], h=h, y=o, **join)
    got = {m: torch.empty_like(t) for m, t in d.items()}
    ds, dc = new(T, 1, c), new(T, c)
    lq.leapquant_block_norm_backward(s[:, None], ds, dh=dh.to(DEV), dy=dy.to(DEV), dres=got["res"], din_weight=got["wi"],
                                     workspace=lq.leapquant_block_norm_workspace(T, 1, c), **join)
    lq.leapquant_scan_backward(plan, where, y, d["dt"], d["A"], d["B"], d["C"], ds[:, 0], dc, got["dt"], got["A"], got["B"],
                               got["C"], dD=got["D"], ddt_bias=got["bias"], dz=got["z"], **more)
    lq.leapquant_conv_backward(where, d["x"], d["w"], dc, got["x"], bias=d["b"], dweight=got["w"], dbias=got["b"],
                               workspace=lq.leapquant_conv_workspace(T, 3, c, 4))
    n = 4 * (9 * 70 + 4 * c + 2 * N + c + 400)
    for m in ref:
        Q.check(got[m], ref[m], n + T, "d" + m)
