"""The recurrence over whole sequences and its gradient on the GPU, against
the 64-bit definition (tests/sequence_reference.py, which also says how the
bounds are derived)."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from oracle import leapquant_oracle as O
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


def make(lengths, hk, hv, dtype=F32, gate="gdn", seed=0, lead=0, tail=0, shift=0.0):
    """Inputs on the host in float64, holding values of their types; `lead`
    tokens before the first sequence and `tail` behind the last are NaN."""
    g = torch.Generator().manual_seed(1000 + seed)
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)  # noqa: E731
    T = lead + sum(lengths) + tail
    cu = [lead]
    for n in lengths:
        cu.append(cu[-1] + n)
    x = {"q": unit(rn(T, hk, 128)), "k": unit(rn(T, hk, 128)), "v": rn(T, hv, 128)}
    x = {n: y.to(dtype) for n, y in x.items()}
    x["beta"] = torch.sigmoid(rn(T, hv)).float()
    x["alpha"] = torch.exp(-torch.nn.functional.softplus(rn(*((T, hv) if gate == "gdn" else (T, hv, 128))) - shift)).float()
    x["S0"] = (0.1 * rn(len(lengths) * hv, 128, 128)).float()
    for n in ("q", "k", "v", "beta", "alpha"):
        x[n][:lead] = float("nan")
        x[n][T - tail:] = float("nan")
    return cu, x


def reference(cu, x, delta=True, state=True, grads=None):
    """64-bit results for the sequences' own tokens (others: zeros)."""
    T, hv = x["v"].shape[:2]
    names = ("q", "k", "v", "beta", "alpha", "S0")
    ins = {n: torch.nan_to_num(x[n].double()) for n in names}
    if not state:
        ins["S0"] = torch.zeros_like(ins["S0"])
    if grads is None:
        return R.recurrence(cu, *[ins[n] for n in names], delta)
    leaves = [ins[n].requires_grad_(True) for n in names]
    o, S = R.recurrence(cu, *leaves, delta)
    do, dS = grads
    loss = (o * torch.nan_to_num(do.double())).sum()
    if dS is not None:
        loss = loss + (S * dS.double()).sum()
    return (o, S, *torch.autograd.grad(loss, leaves, allow_unused=True))


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def forward(cu, x, hk, hv, gate="gdn", delta=True, state=True, save=False, plan=None, stream=None):
    T, n = x["v"].shape[0], (len(cu) - 1) * hv
    d = {m: y.to(DEV) for m, y in x.items()}
    plan = plan or lq.LeapQuantSequence(T, len(cu) - 1, hk, hv, gate, x["q"].dtype, DEV, 0 if delta else lq.LQ_NO_DELTA,
                                        save)
    o = torch.full((T, hv, 128), 7.0, dtype=x["q"].dtype, device=DEV)
    S = torch.full((n, 128, 128), 7.0, device=DEV)
    lq.leapquant_sequence_forward(plan, offsets(cu), d["q"], d["k"], d["v"], d["beta"], d["alpha"], o,
                                  S0=d["S0"] if state else None, S=S, stream=stream)
    return plan, d, o, S


def check_forward(cu, x, o, S, ref, name=""):
    T = max([b - a for a, b in zip(cu, cu[1:])] + [0])
    n = 256 + 3 * T
    ro, rS = ref
    R.check(o[cu[0]:cu[-1]], ro[cu[0]:cu[-1]], n, name + " o")
    R.check(S, rS, n, name + " S")
    # tokens of no sequence are left as they were
    assert (o[:cu[0]] == 7).all() and (o[cu[-1]:] == 7).all(), name


MIXED = [0, 1, 65, 0, 130, 64, 63, 2, 0]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lengths,hk,hv", [([1], 1, 1), ([0], 2, 2), ([5, 0, 1, 16, 3], 2, 4), ([64], 1, 2), ([129], 2, 2),
                                           (MIXED, 2, 6)])
def test_forward(gate, delta, dtype, lengths, hk, hv):
    cu, x = make(lengths, hk, hv, dtype, gate, seed=len(lengths) + hv, lead=3, tail=2)
    _, _, o, S = forward(cu, x, hk, hv, gate, delta)
    check_forward(cu, x, o, S, reference(cu, x, delta))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lengths", [[70], [9, 8, 3], [300, 1]])
def test_forward_from_zero_states(gate, lengths):
    cu, x = make(lengths, 1, 1, BF16, gate, seed=3)
    _, _, o, S = forward(cu, x, 1, 1, gate, state=False)
    check_forward(cu, x, o, S, reference(cu, x, state=False))


@pytest.mark.parametrize("lengths,hk,hv", [([3] * 300, 1, 1), ([2, 1] * 80, 2, 2), ([40] * 70, 1, 4)])
@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_forward_many_sequences(gate, lengths, hk, hv):
    cu, x = make(lengths, hk, hv, BF16, gate, seed=4, shift=2.0)
    _, _, o, S = forward(cu, x, hk, hv, gate)
    check_forward(cu, x, o, S, reference(cu, x))


def special(x, cu):
    """Tokens with decay 0 and 1, strength 0 and 1, zero and repeated keys."""
    T = x["alpha"].shape[0]
    x["alpha"][0:T:7] = 0.0
    x["alpha"][3:T:7] = 1.0
    x["beta"][1:T:5] = 0.0
    x["beta"][2:T:5] = 1.0
    x["k"][4:T:11] = 0.0
    x["k"][6:T:11] = x["k"][5:T:11][: x["k"][6:T:11].shape[0]]
    x["v"][8:T:13] = 0.0


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lengths", [[200], [6, 10]])
def test_forward_special_tokens(gate, lengths):
    cu, x = make(lengths, 1, 2, F32, gate, seed=5)
    special(x, cu)
    _, _, o, S = forward(cu, x, 1, 2, gate)
    check_forward(cu, x, o, S, reference(cu, x))


def test_forward_equal_keys():
    """All keys of a chunk alike: the triangular system at its worst."""
    cu, x = make([200], 1, 1, F32, seed=6)
    x["k"][:] = x["k"][:1]
    x["alpha"][:] = 1.0
    x["beta"][:] = 1.0
    _, _, o, S = forward(cu, x, 1, 1)
    check_forward(cu, x, o, S, reference(cu, x))


def test_in_place_state_and_strided_inputs():
    """S over S0; q, k and v as slices of one projection's rows, o into a wider row, head-major beta and alpha."""
    hk, hv, T = 2, 4, 150
    cu, x = make([100, 50], hk, hv, BF16, seed=7)
    plan = lq.LeapQuantSequence(T, 2, hk, hv, device=DEV)
    rows = torch.zeros((T, 2 * hk + hv + 1, 128), dtype=BF16, device=DEV)
    q, k, v = rows[:, :hk], rows[:, hk:2 * hk], rows[:, 2 * hk:2 * hk + hv]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(x[n])
    wide = torch.full((T, 3 * hv, 128), 7.0, dtype=BF16, device=DEV)
    beta, alpha = (x[n].to(DEV).t().contiguous().t() for n in ("beta", "alpha"))
    S = x["S0"].to(DEV)
    lq.leapquant_sequence_forward(plan, offsets(cu), q, k, v, beta, alpha, wide[:, hv:2 * hv], S0=S, S=S)
    check_forward(cu, x, wide[:, hv:2 * hv], S, reference(cu, x))
    assert (wide[:, :hv] == 7).all() and (wide[:, 2 * hv:] == 7).all()


def test_split_prompt_continues_from_the_state():
    cu, x = make([230], 2, 2, F32, seed=8)
    _, _, o, S = forward(cu, x, 2, 2)
    plan = lq.LeapQuantSequence(230, 1, 2, 2, dtype=F32, device=DEV)
    d = {m: y.to(DEV) for m, y in x.items()}
    state, parts = d["S0"].clone(), []
    for a, b in ((0, 97), (97, 98), (98, 230)):
        o2 = torch.empty((b - a, 2, 128), device=DEV)
        lq.leapquant_sequence_forward(plan, offsets([0, b - a]), *[d[m][a:b] for m in ("q", "k", "v", "beta", "alpha")],
                                      o2, S0=state, S=state)
        parts.append(o2)
    ref = reference(cu, x)
    check_forward(cu, x, torch.cat(parts), state, ref)
    check_forward(cu, x, o, S, ref)


@pytest.mark.parametrize("save", [False, True])
def test_values_that_are_not_finite_stay_in_their_sequence(save):
    cu, x = make([70, 5, 90], 1, 2, F32, seed=9)
    _, _, o, S = forward(cu, x, 1, 2, save=save)
    x["v"][71] = float("nan")
    x["k"][73] = float("inf")
    _, _, o2, S2 = forward(cu, x, 1, 2, save=save)
    keep = torch.ones(165, dtype=torch.bool)
    keep[70:75] = False
    assert torch.equal(o[keep], o2[keep])
    assert torch.equal(S[:2], S2[:2]) and torch.equal(S[4:], S2[4:])


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("cu", [[0, -5, 200, 150], [90, 30, 160, 170], [-100, 500, 500, -1], [170, 160, 100, 0]])
def test_wrong_offsets_stay_inside(gate, cu):
    """Offsets that do not ascend or leave the arrays: unspecified results, but nothing outside is written."""
    _, x = make([160], 1, 1, F32, gate, seed=10)
    plan = lq.LeapQuantSequence(160, 3, 1, 1, gate, F32, DEV)
    guard = torch.full((160 + 256, 1, 128), 7.0, device=DEV)
    states = torch.full((3 + 4, 128, 128), 7.0, device=DEV)
    d = {m: y.to(DEV) for m, y in x.items()}
    lq.leapquant_sequence_forward(plan, offsets(cu), *[d[m] for m in ("q", "k", "v", "beta", "alpha")],
                                  guard[128:288], S=states[2:5])
    torch.cuda.synchronize()
    assert (guard[:128] == 7).all() and (guard[288:] == 7).all()
    assert (states[:2] == 7).all() and (states[5:] == 7).all()


# ---------------------------------------------------------------- gradients
GRADS = ("q", "k", "v", "beta", "alpha", "S0")


def backward(plan, cu, d, do, dS=None, want_state=True, stream=None):
    T, hk, hv = d["v"].shape[0], plan.heads_k, plan.heads_v
    g = {m: torch.full(d[m].shape, 7.0, dtype=d[m].dtype, device=DEV) for m in GRADS[:5]}
    g["S0"] = torch.full(((len(cu) - 1) * hv, 128, 128), 7.0, device=DEV) if want_state else None
    lq.leapquant_sequence_backward(plan, offsets(cu), d["q"], d["k"], d["beta"], d["alpha"], do, g["q"], g["k"], g["v"],
                                   g["beta"], g["alpha"], dS=dS, dS0=g["S0"], stream=stream)
    return g


def check_backward(cu, g, ref):
    T = max([b - a for a, b in zip(cu, cu[1:])] + [0])
    for m, r in zip(GRADS, ref):
        if g[m] is None:
            continue
        r = torch.zeros(g[m].shape, dtype=torch.float64) if r is None else r
        if m == "S0":
            R.check(g[m], r, 768 + 6 * T, "d" + m)
            continue
        R.check(g[m][cu[0]:cu[-1]], r[cu[0]:cu[-1]], 768 + 6 * T, "d" + m)
        assert (g[m][:cu[0]] == 7).all() and (g[m][cu[-1]:] == 7).all(), m


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("lengths,hk,hv", [([1], 1, 1), ([64], 1, 1), ([3, 0, 1, 5], 2, 4), ([129], 2, 2), (MIXED, 2, 6)])
def test_backward(delta, dtype, lengths, hk, hv):
    cu, x = make(lengths, hk, hv, dtype, seed=20 + len(lengths) + hv, lead=3, tail=2)
    g = torch.Generator().manual_seed(77)
    do = torch.randn(x["v"].shape, generator=g).to(dtype)
    dS = 0.3 * torch.randn(x["S0"].shape, generator=g)
    plan, d, o, S = forward(cu, x, hk, hv, "gdn", delta, save=True)
    got = backward(plan, cu, d, do.to(DEV), dS.to(DEV))
    ref = reference(cu, x, delta, grads=(do, dS))
    check_forward(cu, x, o, S, ref[:2])
    check_backward(cu, got, ref[2:])
    # a second backward call on the same workspace gives the same bits
    again = backward(plan, cu, d, do.to(DEV), dS.to(DEV))
    for m in GRADS:
        assert torch.equal(got[m], again[m]), m


@pytest.mark.parametrize("lengths", [[200], [70, 33]])
def test_backward_special_tokens(lengths):
    cu, x = make(lengths, 1, 2, F32, seed=40)
    special(x, cu)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(78))
    plan, d, _, _ = forward(cu, x, 1, 2, save=True)
    check_backward(cu, backward(plan, cu, d, do.to(DEV)), reference(cu, x, grads=(do, None))[2:])


def test_backward_without_states():
    cu, x = make([100, 28], 2, 2, BF16, seed=41)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(79)).to(BF16)
    plan, d, _, _ = forward(cu, x, 2, 2, state=False, save=True)
    got = backward(plan, cu, d, do.to(DEV), want_state=False)
    check_backward(cu, got, reference(cu, x, state=False, grads=(do, None))[2:])


def test_backward_of_no_tokens():
    cu, x = make([0, 0], 1, 2, F32, seed=42)
    plan, d, o, S = forward(cu, x, 1, 2, save=True)
    assert torch.equal(S, d["S0"])
    dS = torch.randn(S.shape, device=DEV)
    got = backward(plan, cu, d, torch.empty((0, 2, 128), device=DEV), dS)
    assert torch.equal(got["S0"], dS)


def test_backward_broadcast_inputs_and_sliced_gradients():
    """One strength for all heads and one do for all tokens (stride 0); gradients into slices of one row; dS0 over dS."""
    hk, hv, T = 2, 2, 90
    cu, x = make([60, 30], hk, hv, F32, seed=43)
    x["beta"] = x["beta"][:, :1].expand(T, hv)
    do = torch.randn((1, hv, 128), generator=torch.Generator().manual_seed(80)).expand(T, hv, 128)
    dS = torch.randn(x["S0"].shape, generator=torch.Generator().manual_seed(81))
    d = {m: y.to(DEV) for m, y in x.items()}
    d["beta"] = x["beta"][:, :1].to(DEV).expand(T, hv)
    plan = lq.LeapQuantSequence(T, 2, hk, hv, dtype=F32, device=DEV, save=True)
    o, S = torch.empty((T, hv, 128), device=DEV), torch.empty_like(d["S0"])
    ins = [d[m] for m in ("q", "k", "v", "beta", "alpha")]
    lq.leapquant_sequence_forward(plan, offsets(cu), *ins, o, S0=d["S0"], S=S)
    rows = torch.full((T, 2 * hk + hv + 2, 128), 7.0, device=DEV)
    gates = torch.full((T, 2 * hv), 7.0, device=DEV)
    g = {"q": rows[:, :hk], "k": rows[:, hk:2 * hk], "v": rows[:, 2 * hk:2 * hk + hv], "beta": gates[:, :hv],
         "alpha": gates[:, hv:], "S0": dS.to(DEV)}
    lq.leapquant_sequence_backward(plan, offsets(cu), d["q"], d["k"], d["beta"], d["alpha"],
                                   do[:1].to(DEV).expand(T, hv, 128), *[g[m] for m in GRADS[:5]], dS=g["S0"],
                                   dS0=g["S0"])
    check_backward(cu, g, reference(cu, x, grads=(do, dS))[2:])
    assert (rows[:, 2 * hk + hv:] == 7).all()


def test_gradient_against_differences_of_the_kernel():
    """Directional differences of the forward kernel (fp32): truncation of a
    central difference is h^2 / 6 of third derivatives (h = 2^-7: 1e-5 of the
    sums), rounding 2^-24 (256 + 3 T) / h of the loss's terms, so 1% of the
    directional derivative's terms is a safe bound."""
    hk, hv, cu = 1, 2, [0, 80, 100]
    _, x = make([80, 20], hk, hv, F32, seed=44, shift=1.0)
    g = torch.Generator().manual_seed(82)
    do, dS = torch.randn(x["v"].shape, generator=g), 0.1 * torch.randn(x["S0"].shape, generator=g)
    plan, d, _, _ = forward(cu, x, hk, hv, save=True)
    grads = backward(plan, cu, d, do.to(DEV), dS.to(DEV))

    def loss(y):
        _, _, o, S = forward(cu, y, hk, hv)
        return (o.double().cpu() * do).sum() + (S.double().cpu() * dS).sum()

    h = 2.0 ** -7
    for m in GRADS:
        v = torch.randn(x[m].shape, generator=g)
        v = v / v.norm() * x[m].norm()
        num = (loss({**x, m: x[m] + h * v}) - loss({**x, m: x[m] - h * v})) / (2 * h)
        terms = grads[m].double().cpu() * v
        assert abs(num - terms.sum()) <= 0.01 * terms.norm() * terms.numel() ** 0.5, m


# ---------------------------------------------------------------- streams, graphs, together
def test_streams_and_a_plan_each():
    cu, x = make([150, 40], 2, 4, BF16, seed=50)
    _, _, o, S = forward(cu, x, 2, 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(forward(cu, x, 2, 4, stream=s))
    torch.cuda.synchronize()
    for _, _, o2, S2 in outs:
        assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("lengths", [[130, 20, 0], [3, 2, 1]])
def test_captured_step(lengths):
    """Forward and backward captured once, replayed with new inputs and other work between, equal the eager calls."""
    hk, hv = 2, 4
    sets = [make(lengths, hk, hv, BF16, seed=60 + i) for i in range(3)]
    cu = sets[0][0]
    T = cu[-1]
    plan = lq.LeapQuantSequence(T, len(lengths), hk, hv, dtype=BF16, device=DEV, save=True)
    serve = lq.LeapQuantSequence(T, len(lengths), hk, hv, dtype=BF16, device=DEV)
    ins = {m: y.to(DEV).clone() for m, y in sets[0][1].items()}
    at, do = offsets(cu), torch.randn((T, hv, 128), device=DEV).to(BF16)
    out = {m: torch.empty_like(ins[m]) for m in GRADS}
    o, o2, S = torch.empty_like(ins["v"]), torch.empty_like(ins["v"]), torch.empty_like(ins["S0"])
    names = ("q", "k", "v", "beta", "alpha")

    def step():
        lq.leapquant_sequence_forward(plan, at, *[ins[m] for m in names], o, S0=ins["S0"], S=S)
        lq.leapquant_sequence_backward(plan, at, ins["q"], ins["k"], ins["beta"], ins["alpha"], do,
                                       *[out[m] for m in GRADS[:5]], dS=S, dS0=out["S0"])
        lq.leapquant_sequence_forward(serve, at, *[ins[m] for m in names], o2, S0=ins["S0"])

    def results():
        return [t.clone() for t in (o, o2, S, *out.values())]

    eager = []
    for _, x in sets:
        for m in ins:
            ins[m].copy_(x[m])
        step()
        eager.append(results())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in (0, 1, 2, 1, 0):
        for m in ins:
            ins[m].copy_(sets[i][1][m])
        for t in (o, o2, S, *out.values()):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results(), eager[i]):
            assert torch.equal(a, b)
        (torch.randn(512, 512, device=DEV) @ torch.randn(512, 512, device=DEV)).sum().item()


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_prompt_then_decode(gate):
    """Projections -> head norm -> prompt -> quantized state -> a window of
    decoded tokens, against the 64-bit forms and the decode oracle."""
    hk = hv = 2
    p, r, T = 8, 4, 75
    lengths = [40, 35]
    cu, x = make(lengths, hk, hv, BF16, gate, seed=70)
    g = torch.Generator().manual_seed(83)
    raw = {m: (3 * torch.randn((T, hk, 128), generator=g)).to(BF16) for m in ("q", "k")}
    pos = torch.cat([torch.arange(n) for n in lengths])
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    q, k = (torch.empty((T, hk, 128), dtype=F32, device=DEV) for _ in range(2))
    lq.leapquant_head_norm(raw["q"].to(DEV), raw["k"].to(DEV), q, k, q_scale=128 ** -0.5, positions=pos.to(DEV),
                           inv_freq=freq.to(DEV))
    for m, y, scale in (("q", q, 128 ** -0.5), ("k", k, 1.0)):
        R.check(y, R.head_norm(raw[m].double(), "l2", 1e-6, None, scale, pos, freq, False), 160, m)
    x = {**x, "q": q.cpu(), "k": k.cpu(), "v": x["v"].float()}
    _, _, o, S = forward(cu, x, hk, hv, gate, state=False)
    check_forward(cu, x, o, S, reference(cu, x, state=False))
    n = len(lengths) * hv
    st = lq.LeapQuantState(n, p, r, gate, DEV)
    lq.leapquant_quantize_state(st, S)
    tok = {m: torch.randn((p, n, 128), generator=g) for m in ("q", "k", "v")}
    tok["q"], tok["k"] = (tok[m] / tok[m].norm(dim=-1, keepdim=True) for m in ("q", "k"))
    tok["beta"] = torch.sigmoid(torch.randn((p, n), generator=g))
    tok["alpha"] = torch.sigmoid(torch.randn((p, n) if gate == "gdn" else (p, n, 128), generator=g))
    out = torch.empty((p, n, 128), device=DEV)
    for t in range(p):
        lq.leapquant_decode_step(st, t, *[tok[m][t].to(DEV) for m in ("q", "k", "v", "beta", "alpha")], out[t])
    want, _ = O.run_windowed(S.cpu().numpy(), {m: y.numpy().astype("float64") for m, y in tok.items()}, p, r,
                             O.GATE_GDN if gate == "gdn" else O.GATE_KDA)
    want = torch.as_tensor(want)
    assert ((out.cpu() - want).abs() <= 1e-4 + 1e-3 * want.abs()).all()  # the decode calls' own bounds


def test_few_tokens_equal_the_dense_steps():
    """A sequence of one token each is the dense fp32 step of the baselines."""
    n = 40
    cu, x = make([1] * n, 1, 1, F32, seed=71)
    _, d, o, S = forward(cu, x, 1, 1)
    S2, o2 = d["S0"].clone(), torch.empty((n, 128), device=DEV)
    lq.leapquant_dense_step(S2, "gdn", d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["beta"][:, 0].contiguous(),
                            d["alpha"][:, 0].contiguous(), o2)
    ref = reference(cu, x)
    check_forward(cu, x, o, S, ref)
    R.check(o2, ref[0][:, 0], 259, "dense o")
    R.check(S2, ref[1], 259, "dense S")


def test_training_chain():
    """Head norm -> sequence -> its gradient -> the norm's gradient, against
    automatic differentiation of the 64-bit forms through all of it."""
    hk, hv, T, cu = 2, 4, 110, [0, 70, 110]
    _, x = make([70, 40], hk, hv, F32, seed=72, shift=2.0)
    g = torch.Generator().manual_seed(84)
    raw = {m: torch.randn((T, hk, 128), generator=g) for m in ("q", "k")}
    w = {m: 1 + 0.1 * torch.randn(128, generator=g) for m in ("q", "k")}
    do = torch.randn((T, hv, 128), generator=g)
    pos, freq = torch.arange(T) + 1000, 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    dev = lambda t: t.to(DEV)  # noqa: E731
    how = dict(norm="rms", eps=1e-5, q_weight=dev(w["q"]), k_weight=dev(w["k"]), q_scale=0.01, positions=dev(pos),
               inv_freq=dev(freq), interleaved=True)
    # RMS keys have norm sqrt(128): divided by it through the weight, to be unit keys
    how["k_weight"] = how["k_weight"] * 128 ** -0.5
    qr, kr = dev(raw["q"]), dev(raw["k"])
    q, k = torch.empty_like(qr), torch.empty_like(kr)
    lq.leapquant_head_norm(qr, kr, q, k, **how)
    plan, d, o, S = forward(cu, {**x, "q": q.cpu(), "k": k.cpu()}, hk, hv, state=False, save=True)
    gr = backward(plan, cu, d, dev(do), want_state=False)
    dqr, dkr, dwq, dwk = (torch.empty_like(t) for t in (qr, kr, how["q_weight"], how["k_weight"]))
    ws = lq.leapquant_head_norm_workspace(T, hk, hk)
    lq.leapquant_head_norm_backward(qr, kr, gr["q"], gr["k"], dqr, dkr, dq_weight=dwq, dk_weight=dwk, workspace=ws,
                                    **how)
    leaves = [t.double().cpu().requires_grad_(True) for t in (qr, kr, how["q_weight"], how["k_weight"])]
    qq = R.head_norm(leaves[0], "rms", 1e-5, leaves[2], 0.01, pos, freq, True)
    kk = R.head_norm(leaves[1], "rms", 1e-5, leaves[3], 1.0, pos, freq, True)
    oo, _ = R.recurrence(cu, qq, kk, x["v"].double(), x["beta"].double(), x["alpha"].double(),
                         torch.zeros(x["S0"].shape, dtype=torch.float64))
    ref = torch.autograd.grad((oo * do).sum(), leaves)
    # the chain of the sequence's gradient, the norm's 160, and for the weights a sum over T tokens and their heads
    n = 768 + 6 * 70 + 2 * 160
    for got, want, more, name in ((dqr, ref[0], 0, "q"), (dkr, ref[1], 0, "k"), (dwq, ref[2], T * hk, "wq"),
                                  (dwk, ref[3], T * hk, "wk")):
        R.check(got, want, n + more, name)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_long_sequence(gate):
    """Thousands of tokens from a state: errors do not pile up beyond the bound (reference on the GPU, 64 bits)."""
    T, hk, hv = 2500, 1, 2
    cu, x = make([T], hk, hv, F32, gate, seed=90, shift=4.0)
    _, _, o, S = forward(cu, x, hk, hv, gate)
    names = ("q", "k", "v", "beta", "alpha", "S0")
    ro, rS = R.recurrence(cu, *[x[m].double().to(DEV) for m in names])
    check_forward(cu, x, o, S, (ro, rS))


def test_long_backward():
    T, hk, hv = 1000, 1, 2
    cu, x = make([T], hk, hv, F32, seed=91, shift=4.0)
    g = torch.Generator().manual_seed(92)
    do, dS = torch.randn(x["v"].shape, generator=g), torch.randn(x["S0"].shape, generator=g)
    plan, d, _, _ = forward(cu, x, hk, hv, save=True)
    got = backward(plan, cu, d, do.to(DEV), dS.to(DEV))
    leaves = [x[m].double().to(DEV).requires_grad_(True) for m in GRADS]
    o, S = R.recurrence(cu, *leaves)
    ref = torch.autograd.grad((o * do.double().to(DEV)).sum() + (S * dS.double().to(DEV)).sum(), leaves)
    check_backward(cu, got, ref)


@pytest.mark.parametrize("lengths", [[70], [2, 3]])
def test_offsets_past_32_bits(lengths):
    """v and o with tokens 2^26 elements apart: offsets of more than 2^32 bytes."""
    T, step = sum(lengths), 1 << 26
    cu, x = make(lengths, 1, 1, BF16, seed=93)
    far = torch.empty(T * step, dtype=BF16, device=DEV)
    v, o = (far.as_strided((T, 1, 128), (step, 128, 1), at) for at in (0, 1024))
    v.copy_(x["v"])
    plan = lq.LeapQuantSequence(T, len(lengths), 1, 1, device=DEV)
    d = {m: y.to(DEV) for m, y in x.items()}
    S = torch.empty_like(d["S0"])
    lq.leapquant_sequence_forward(plan, offsets(cu), d["q"], d["k"], v, d["beta"], d["alpha"], o, S0=d["S0"], S=S)
    check_forward(cu, x, o, S, reference(cu, x))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lengths", [[80, 7], [5, 4]])
def test_head_major_arrays(gate, lengths):
    """[heads, tokens, 128] arrays, seen as [tokens, heads, 128]."""
    hk, hv, T = 2, 4, sum(lengths)
    cu, x = make(lengths, hk, hv, F16, gate, seed=94)
    turn = lambda t: t.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    d = {m: (y.to(DEV) if m == "S0" else turn(y)) for m, y in x.items()}
    plan = lq.LeapQuantSequence(T, 2, hk, hv, gate, F16, DEV)
    o, S = turn(torch.full((T, hv, 128), 7.0, dtype=F16)), torch.empty_like(d["S0"])
    lq.leapquant_sequence_forward(plan, offsets(cu), *[d[m] for m in ("q", "k", "v", "beta", "alpha")], o, S0=d["S0"],
                                  S=S)
    check_forward(cu, x, o, S, reference(cu, x))


def test_one_plan_for_calls_of_many_sizes():
    """A plan's workspace serves every smaller call, whichever form it takes."""
    plan = lq.LeapQuantSequence(300, 40, 1, 2, dtype=F32, device=DEV)
    for i, lengths in enumerate(([300], [1] * 40, [7] * 40, [30] * 10, [25], [24], [0, 25, 0], [150, 150], [26] * 11)):
        cu, x = make(lengths, 1, 2, F32, seed=100 + i)
        _, _, o, S = forward(cu, x, 1, 2, plan=plan)
        check_forward(cu, x, o, S, reference(cu, x))


def test_many_value_heads_for_a_key_head():
    cu, x = make([66, 30], 1, 8, BF16, seed=110)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(111)).to(BF16)
    plan, d, o, S = forward(cu, x, 1, 8, save=True)
    ref = reference(cu, x, grads=(do, None))
    check_forward(cu, x, o, S, ref[:2])
    check_backward(cu, backward(plan, cu, d, do.to(DEV)), ref[2:])


MANY = [1, 0, 64, 64, 130, 37, 5, 0, 90, 17] * 4  # equal, empty and the longest in the middle


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lengths", [MANY, MANY + [70] * 25, [0] * 39 + [1100]])
def test_more_workgroups_than_the_chip_holds(gate, lengths):
    """Scans whose grid begins with the longest sequences, and (more than 64 sequences) in their order."""
    cu, x = make(lengths, 2, 4, BF16, gate, seed=114, shift=2.0)
    _, _, o, S = forward(cu, x, 2, 4, gate)
    check_forward(cu, x, o, S, reference(cu, x))


@pytest.mark.parametrize("lengths", [MANY, MANY + [33] * 25])
def test_backward_of_more_workgroups_than_the_chip_holds(lengths):
    cu, x = make(lengths, 2, 4, BF16, seed=115, shift=2.0)
    g = torch.Generator().manual_seed(116)
    do, dS = torch.randn(x["v"].shape, generator=g).to(BF16), torch.randn(x["S0"].shape, generator=g)
    plan, d, o, S = forward(cu, x, 2, 4, save=True)
    ref = reference(cu, x, grads=(do, dS))
    check_forward(cu, x, o, S, ref[:2])
    check_backward(cu, backward(plan, cu, d, do.to(DEV), dS.to(DEV)), ref[2:])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_results_repeat_and_gradients_may_lie_over_states(dtype):
    """The same call again gives the same bits; a second backward call on one workspace too, with dS0 in dS."""
    cu, x = make([150, 0, 31, 64], 2, 4, dtype, seed=117, shift=2.0)
    g = torch.Generator().manual_seed(118)
    do, dS = torch.randn(x["v"].shape, generator=g).to(DEV, dtype), torch.randn(x["S0"].shape, generator=g).to(DEV)
    plan, d, o, S = forward(cu, x, 2, 4, save=True)
    first = backward(plan, cu, d, do, dS)
    again = {m: torch.empty_like(y) for m, y in first.items()}
    again["S0"] = dS.clone()
    lq.leapquant_sequence_backward(plan, offsets(cu), d["q"], d["k"], d["beta"], d["alpha"], do, *[again[m] for m in GRADS[:5]],
                                   dS=again["S0"], dS0=again["S0"])
    for m in GRADS:
        assert torch.equal(first[m], again[m]), m
    _, _, o2, S2 = forward(cu, x, 2, 4, save=True, plan=plan)
    assert torch.equal(o, o2) and torch.equal(S, S2)


def test_gradients_of_values_that_are_not_finite_stay_in_their_sequence():
    cu, x = make([70, 5, 90], 1, 2, F32, seed=112)
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(113)).to(DEV)
    runs = []
    for bad in (False, True):
        if bad:
            x["v"][71] = float("nan")
        plan, d, _, _ = forward(cu, x, 1, 2, save=True)
        y = do.clone()
        if bad:
            y[73] = float("inf")
        runs.append(backward(plan, cu, d, y))
    keep = torch.ones(165, dtype=torch.bool)
    keep[70:75] = False
    for m in GRADS[:5]:
        assert torch.equal(runs[0][m][keep], runs[1][m][keep]), m
    assert torch.equal(runs[0]["S0"][:2], runs[1]["S0"][:2]) and torch.equal(runs[0]["S0"][4:], runs[1]["S0"][4:])


def test_refusals_on_the_device():
    plan = lq.LeapQuantSequence(10, 2, 2, 4, dtype=F32, device=DEV)
    z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    q, v, b, cu = z(10, 2, 128), z(10, 4, 128), z(10, 4), offsets([0, 4, 10])
    ok = dict(cu_seqlens=cu, q=q, k=q, v=v, beta=b, alpha=b, o=z(10, 4, 128))
    lq.leapquant_sequence_forward(plan, **ok)
    bad = [dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu.cpu()), dict(q=z(10, 2, 64)), dict(k=z(9, 2, 128)),
           dict(v=v.half()), dict(alpha=z(10, 4, 128)), dict(beta=z(10, 2)), dict(o=z(10, 4, 128).cpu()),
           dict(q=z(10, 128, 2).transpose(1, 2)), dict(S=z(3, 128, 128)), dict(S0=z(8, 128, 128).double()),
           dict(cu_seqlens=offsets([0, 1, 2, 10])), dict(q=z(11, 2, 128))]
    for kw in bad:
        with pytest.raises(ValueError):
            lq.leapquant_sequence_forward(plan, **{**ok, **kw})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_sequence_forward(plan, **{**ok, "o": v})
    S = z(8 * 128 * 128 + 64)
    with pytest.raises(lq.LeapQuantError):  # states that overlap in part
        lq.leapquant_sequence_forward(plan, **ok, S0=S[:8 * 128 * 128].view(8, 128, 128),
                                      S=S[64:].view(8, 128, 128))
