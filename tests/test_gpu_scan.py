"""The selective scan on the GPU against its 64-bit form.  Roundings are counted
in tests/layer_reference.py: n = 4 T + 32 (states), 4 T + N + 64 (outputs),
9 T + 2 N + per + 160 (gradients) of the sums of absolute terms."""
import pytest
import torch

import recurrent_state_quant_amd as lq
from tests import layer_reference as R
from tests.sequence_reference import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
LOW = ("x", "dt", "B", "C", "z")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    lq.load()
    yield
    torch.cuda.synchronize()


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def make(cu, tokens, c, N, G, dtype, gate=True, weights=True, state=True, seed=0, slow=0.0):
    """slow: moves the steps; negative ones make small steps, that is long memories."""
    g = torch.Generator().manual_seed(700 + seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    n = len(cu) - 1
    x = {"x": r(tokens, c), "dt": 0.5 * r(tokens, c) + (0 if weights else slow), "B": r(tokens, G, N), "C": r(tokens, G, N),
         "z": r(tokens, c) if gate else None, "dy": r(tokens, c)}
    x = {m: None if t is None else t.to(dtype) for m, t in x.items()}
    x["A"] = -torch.arange(1, N + 1) * torch.exp(0.1 * r(c, N))
    x["D"], x["bias"] = (1 + 0.1 * r(c), r(c) + slow) if weights else (None, None)
    x["S0"], x["dS"] = (r(n, c, N), r(n, c, N)) if state else (None, None)
    return x


def dev(x):
    return {m: None if t is None else t.to(DEV) for m, t in x.items()}


def reference(cu, x, softplus=True):
    """(results, sums of absolute terms) of the 64-bit form, forward and backward."""
    n, (c, N) = len(cu) - 1, x["A"].shape
    v = {m: None if t is None else t.double() for m, t in x.items()}
    for m in ("S0", "dS"):
        v[m] = torch.zeros((n, c, N), dtype=torch.float64) if v[m] is None else v[m]
    args = [v[m] for m in ("x", "dt", "A", "B", "C", "D", "bias", "z", "S0", "dy", "dS")]
    return tuple(R.scan_adjoint(cu, *args, softplus=softplus, absolute=a) for a in (False, True))


def weights(d):
    return dict(D=d["D"], dt_bias=d["bias"], z=d["z"])


def forward(cu, d, save=False, plan=None, softplus=True, y=None, S=None):
    tokens, c = d["x"].shape
    N, G = d["A"].shape[1], d["B"].shape[1]
    if plan is None:
        plan = lq.LeapQuantScan(tokens, len(cu) - 1, c, N, groups=G, dtype=d["x"].dtype, softplus=softplus, save=save)
        plan.workspace.fill_(255)  # NaN wherever it is read unwritten
    y = torch.full((tokens, c), 7.0, dtype=d["x"].dtype, device=DEV) if y is None else y
    S = torch.full((len(cu) - 1, c, N), 7.0, device=DEV) if S is None else S
    lq.leapquant_scan_forward(plan, offsets(cu), d["x"], d["dt"], d["A"], d["B"], d["C"], y, S0=d["S0"], S=S, **weights(d))
    return plan, y, S


def backward(plan, cu, d, dS0=None):
    out = {m: torch.full_like(d[m], 7.0) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z") if d[m] is not None}
    out["S0"] = torch.full((len(cu) - 1, *d["A"].shape), 7.0, device=DEV) if dS0 is None else dS0
    lq.leapquant_scan_backward(plan, offsets(cu), d["x"], d["dt"], d["A"], d["B"], d["C"], d["dy"], out["x"], out["dt"],
                               out["A"], out["B"], out["C"], dD=out.get("D"), ddt_bias=out.get("bias"), dz=out.get("z"),
                               dS=d["dS"], dS0=out["S0"], **weights(d))
    return out


def covered(cu, tokens):
    keep = torch.zeros(tokens, dtype=torch.bool)
    keep[cu[0]:cu[-1]] = True
    return keep


def check_all(cu, d, x, y, S, out=None, softplus=True):
    tokens, (c, N) = d["x"].shape[0], x["A"].shape
    ref, top = reference(cu, x, softplus)
    keep = covered(cu, tokens)
    T = max([b - a for a, b in zip(cu, cu[1:])] + [0])
    check(y.cpu()[keep], ref["y"][keep], 4 * T + N + 64, "y", top["y"][keep])
    check(S, ref["S"], 4 * T + 32, "S", top["S"])
    assert (y.cpu()[~keep] == 7).all()
    if out is None:
        return
    n = 9 * T + 2 * N + c // x["B"].shape[1] + 160
    for m, t in out.items():
        t = t.cpu()
        if m in LOW:
            assert (t[~keep] == 7).all(), m
            check(t[keep], ref[m][keep], n, "d" + m, top[m][keep])
        else:
            check(t, ref[m], n + (0 if m == "S0" else tokens), "d" + m, top[m])


CASES = [([0, 1], 1, 1, 16, 1), ([0, 5, 5, 12], 12, 64, 8, 1), ([2, 9, 75], 80, 70, 16, 2), ([0, 0, 31, 64, 200], 200, 96, 16, 1),
         ([3, 3, 3], 6, 24, 8, 4), ([0, 33, 34, 36, 39, 43, 160], 161, 40, 32, 1), ([0, 300], 300, 130, 32, 2),
         ([0, 8, 16, 24, 88], 88, 520, 8, 2), ([0, 257], 257, 300, 16, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("cu,tokens,c,N,G", CASES)
def test_scan_and_gradient(cu, tokens, c, N, G, dtype):
    gate, plain, state = tokens % 2 == 0, tokens % 3 == 0, tokens != 300
    x = make(cu, tokens, c, N, G, dtype, gate, not plain, state, seed=tokens, slow=-2.0 if c % 4 else 0.0)
    d = dev(x)
    _, y, S = forward(cu, d)
    check_all(cu, d, x, y, S)
    plan, y2, S2 = forward(cu, d, save=True)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    check_all(cu, d, x, y, S, backward(plan, cu, d))


@pytest.mark.parametrize("N", [8, 16, 32])
def test_steps_as_they_are(N):
    """Without the softplus, also steps of zero."""
    cu = [0, 20, 70]
    x = make(cu, 70, 48, N, 1, F32, seed=N)
    x["dt"] = x["dt"].abs()
    x["bias"] = None
    x["dt"][5] = 0.0
    d = dev(x)
    plan, y, S = forward(cu, d, save=True, softplus=False)
    check_all(cu, d, x, y, S, backward(plan, cu, d), softplus=False)


@pytest.mark.parametrize("v", [-1e4, -80.0, -20.0, -3.0, 0.0, 3.0, 20.0, 90.0, 1e4])
def test_steps_far_from_zero(v):
    """Steps of inputs far below zero keep their relative accuracy, those far above are their input; an input of minus
    infinity is a step of zero."""
    cu, c = [0, 3], 64
    x = make(cu, 3, c, 8, 1, F32, gate=False, weights=False, state=False, seed=20)
    x["dt"] = v * (1 + 0.1 * torch.rand((3, c), generator=torch.Generator().manual_seed(1)))
    x["dt"][1] = float("-inf")
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    ref, top = reference(cu, x)
    assert torch.isfinite(y).all()
    # n roundings of each state's own terms (top), not of the tensor's largest.  e^-|v| below the normal range, 2^-126,
    # is zero on the device: a step may be off by that, and a state by that times two tokens' |x B| <= 4 * 4 each
    assert x["x"].abs().max() <= 4 and x["B"].abs().max() <= 4
    off = (S.cpu().double() - ref["S"]).abs()
    assert (off <= (4 * 3 + 32) * 2.0 ** -24 * top["S"] + 32 * 2.0 ** -126).all()
    grads = backward(plan, cu, d)
    assert (grads["dt"][1] == 0).all() and all(torch.isfinite(t).all() for t in grads.values())


def test_many_chunks():
    """One sequence of many chunks beside short ones, and long memories."""
    cu = [0, 3, 3, 1400, 1431]
    x = make(cu, 1431, 64, 16, 1, F32, seed=21, slow=-5.0)
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    check_all(cu, d, x, y, S, backward(plan, cu, d))


def test_more_channels_than_one_pass_holds():
    """Longer chunks where channels alone fill the chip (against the same scan in pieces of 64 channels)."""
    cu, c = [0, 700, 900], 1 << 15
    g = torch.Generator(device=DEV).manual_seed(22)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    d = {"x": r(900, c), "dt": r(900, c) - 2, "z": r(900, c), "dy": r(900, c), "B": r(900, 1, 8), "C": r(900, 1, 8),
         "A": -torch.rand((c, 8), generator=g, device=DEV) * 4, "D": r(c), "bias": r(c), "S0": r(2, c, 8), "dS": r(2, c, 8)}
    plan, y, S = forward(cu, d, save=True)
    out = backward(plan, cu, d)
    pick = torch.arange(64, device=DEV) * (c // 64)
    part = {m: t[:, pick].contiguous() if m in ("x", "dt", "z", "dy", "S0", "dS") else t[pick] if m in ("A", "D", "bias") else t
            for m, t in d.items()}
    x = {m: t.cpu() for m, t in part.items()}
    ref, top = reference(cu, x)
    n = 9 * 700 + 16 + 64 + 160
    check(y[:, pick], ref["y"], n, "y", top["y"])
    check(S[:, pick], ref["S"], n, "S", top["S"])
    for m in ("x", "dt", "z"):
        check(out[m][:, pick], ref[m], n, m, top[m])
    check(out["S0"][:, pick], ref["S0"], n, "S0", top["S0"])
    for m in ("A", "D", "bias"):
        check(out[m][pick], ref[m], n + 900, m, top[m])


def test_states_in_place_and_results_that_repeat():
    cu = [0, 40, 40, 45, 245]
    x = make(cu, 245, 96, 16, 2, BF16, seed=23)
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    first = backward(plan, cu, d)
    again = backward(plan, cu, d)
    over = d["dS"].clone()
    third = backward(plan, cu, {**d, "dS": over}, dS0=over)
    for m in first:
        assert torch.equal(first[m], again[m]) and torch.equal(first[m], third[m]), m
    states = d["S0"].clone()
    _, y2, S2 = forward(cu, {**d, "S0": states}, S=states)
    assert torch.equal(y, y2) and torch.equal(S, S2)


def test_one_plan_for_many_sizes():
    plan = lq.LeapQuantScan(1000, 5, 64, 16, dtype=F32, save=True)
    for k, cu in enumerate(([0, 1000], [0, 3], [0, 1, 2, 3, 4, 5], [0, 0], [0, 500, 999])):
        tokens = cu[-1]
        x = make(cu, tokens, 64, 16, 1, F32, seed=30 + k)
        d = dev(x)
        plan.workspace.fill_(255)
        _, y, S = forward(cu, d, plan=plan)
        check_all(cu, d, x, y, S, backward(plan, cu, d))
    with pytest.raises(ValueError, match="holds a forward"):
        backward(plan, [0, 499, 998], dev(make([0, 499, 998], 998, 64, 16, 1, F32)))
    with pytest.raises(ValueError, match="plan is for"):
        forward([0, 1001], dev(make([0, 1001], 1001, 64, 16, 1, F32)), plan=plan)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,c,N,G", [(1, 1, 16, 1), (5, 64, 8, 2), (37, 130, 32, 1), (64, 1000, 16, 4)])
def test_step(rows, c, N, G, dtype):
    """Slots in any order, some rows idle, the other slots left as they are; in place and not."""
    g = torch.Generator().manual_seed(rows)
    n = rows + 3
    x = make([0, rows], rows, c, N, G, dtype, gate=rows != 5, weights=rows != 37, seed=40)
    S = torch.randn((n, c, N), generator=g)
    slots = torch.randperm(n, generator=g)[:rows].to(torch.int32)
    idle = torch.zeros(rows, dtype=torch.bool)
    if rows > 4:
        slots[1], slots[3] = -1, n
        idle[1] = idle[3] = True
    d = dev(x)
    kw = dict(D=d["D"], dt_bias=d["bias"], z=d["z"], slots=slots.to(DEV))
    y, Sd, out = torch.full_like(d["x"], 7.0), S.to(DEV), torch.full_like(S, 7.0).to(DEV)
    lq.leapquant_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], y, Sd, S_out=out, **kw)
    assert torch.equal(Sd.cpu(), S)
    live = torch.nonzero(~idle).flatten()
    v = {m: None if t is None else t.double() for m, t in x.items()}
    each = list(range(len(live) + 1))
    pick = {m: None if v[m] is None else v[m][live] for m in ("x", "dt", "B", "C", "z")}
    listed = slots[live].long()
    args = [pick["x"], pick["dt"], v["A"], pick["B"], pick["C"], v["D"], v["bias"], pick["z"], S.double()[listed],
            torch.ones_like(pick["x"]), torch.zeros((len(live), c, N), dtype=torch.float64)]
    ref, top = (R.scan_adjoint(each, *args, absolute=a) for a in (False, True))
    check(y.cpu()[live], ref["y"], 4 + N + 64, "y", top["y"])
    check(out.cpu()[listed], ref["S"], 36, "S", top["S"])
    assert (y.cpu()[idle] == 7).all()
    rest = torch.ones(n, dtype=torch.bool)
    rest[listed] = False
    assert (out.cpu()[rest] == 7).all()
    y2 = torch.full_like(y, 7.0)
    lq.leapquant_scan_step(d["x"], d["dt"], d["A"], d["B"], d["C"], y2, Sd, **kw)
    assert torch.equal(y, y2) and torch.equal(Sd[listed.to(DEV)], out[listed.to(DEV)])
    assert torch.equal(Sd.cpu()[rest], S[rest])


def test_a_prompt_and_its_next_tokens():
    """A prompt by chunks, the next tokens by steps, against the whole sequence's 64-bit form."""
    cu, c = [0, 90], 128
    x = make(cu, 90, c, 16, 1, F32, seed=41)
    d = dev(x)
    ref, top = reference(cu, x)
    head = {m: d[m][:70] if m in ("x", "dt", "B", "C", "z", "dy") else d[m] for m in d}
    _, y, S = forward([0, 70], head)
    check(y, ref["y"][:70], 4 * 70 + 80, "y", top["y"][:70])
    for t in range(70, 90):
        yt = torch.empty((1, c), device=DEV)
        lq.leapquant_scan_step(*[d[m][t:t + 1] if m != "A" else d[m] for m in ("x", "dt", "A", "B", "C")], yt, S, D=d["D"],
                               dt_bias=d["bias"], z=d["z"][t:t + 1])
        check(yt, ref["y"][t:t + 1], 4 * 90 + 80, "y", top["y"][t:t + 1])
    check(S, ref["S"], 4 * 90 + 32, "S", top["S"])


def test_slices_of_projections():
    """x and z out of one row, dt, B and C out of another, gradients into slices: the same results."""
    cu, c, N, G = [0, 30, 100], 72, 16, 2
    x = make(cu, 100, c, N, G, BF16, seed=42)
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    first = backward(plan, cu, d)
    rows = torch.full((100, 2 * c + 3), 9.0, dtype=BF16, device=DEV)
    low = torch.full((100, 40 + 2 * G * N), 9.0, dtype=BF16, device=DEV)
    s = {**d, "x": rows[:, 1:c + 1], "z": rows[:, c + 2:2 * c + 2], "B": low[:, 40:40 + G * N].unflatten(1, (G, N)),
         "C": low[:, 40 + G * N:].unflatten(1, (G, N))}
    for m in ("x", "z", "B", "C"):
        s[m].copy_(d[m])
    plan2, y2, S2 = forward(cu, s, save=True)
    assert torch.equal(y, y2) and torch.equal(S, S2)
    grow, glow = torch.full_like(rows, 9.0), torch.full_like(low, 9.0)
    out = {m: torch.empty_like(first[m]) for m in ("dt", "A", "D", "bias", "S0")}
    out |= {"x": grow[:, 1:c + 1], "z": grow[:, c + 2:2 * c + 2], "B": glow[:, 40:40 + G * N].unflatten(1, (G, N)),
            "C": glow[:, 40 + G * N:].unflatten(1, (G, N))}
    lq.leapquant_scan_backward(plan2, offsets(cu), s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], out["x"], out["dt"],
                               out["A"], out["B"], out["C"], dD=out["D"], ddt_bias=out["bias"], dz=out["z"], dS=s["dS"],
                               dS0=out["S0"], **weights(s))
    for m in first:
        assert torch.equal(first[m], out[m]), m
    assert (grow[:, 0] == 9).all() and (grow[:, c + 1] == 9).all() and (grow[:, -1] == 9).all() and (glow[:, :40] == 9).all()


def test_far_offsets():
    """Element offsets beyond 2^31."""
    T, c, stride = 600, 64, 4_000_000
    d = dev(make([0, T], T, c, 16, 1, BF16, seed=43))
    far = lambda: torch.empty(T * stride, dtype=BF16, device=DEV).as_strided((T, c), (stride, 1))  # noqa: E731
    s = {**d, "x": far(), "z": far()}
    for m in ("x", "z"):
        s[m].copy_(d[m])
    _, y, S = forward([0, T], d)
    _, y2, S2 = forward([0, T], s, y=far())
    assert torch.equal(y, y2) and torch.equal(S, S2)


def test_values_that_are_not_finite_stay_in_their_channel_and_sequence():
    cu = [0, 70, 75, 165]
    x = make(cu, 165, 80, 16, 1, F32, seed=44)
    runs = []
    for bad in (False, True):
        if bad:
            x["x"][71, 3] = float("nan")
            x["dy"][73, 5] = float("inf")
        d = dev(x)
        plan, y, S = forward(cu, d, save=True)
        runs.append((y, S, backward(plan, cu, d)))
    (y0, S0, g0), (y1, S1, g1) = runs
    rows = torch.ones(165, dtype=torch.bool, device=DEV)
    rows[70:75] = False
    chans = torch.ones(80, dtype=torch.bool, device=DEV)
    chans[3] = chans[5] = False
    assert torch.equal(y0[rows], y1[rows]) and torch.equal(y0[:, chans], y1[:, chans])
    assert torch.equal(S0[:, chans], S1[:, chans]) and torch.equal(S0[[0, 2]], S1[[0, 2]])
    for m in ("x", "dt", "z"):
        assert torch.equal(g0[m][rows], g1[m][rows]) and torch.equal(g0[m][:, chans], g1[m][:, chans]), m
    for m in ("B", "C"):
        assert torch.equal(g0[m][rows], g1[m][rows]), m
    for m in ("A", "D", "bias"):
        assert torch.equal(g0[m][chans], g1[m][chans]), m


def test_offsets_that_do_not_ascend_stay_in_bounds():
    """Unspecified results, but no access outside the arrays (offsets are held to [0, tokens])."""
    d = dev(make([0, 40, 80, 120], 120, 64, 16, 1, F32, seed=45))
    for cu in ([90, 3, 120, 0], [-5, 1 << 30, 7, 1 << 30], [120, 120, 120, 120], [130, 140, 150, 160]):
        guard = torch.full((3, 120, 64), 7.0, device=DEV)
        plan = lq.LeapQuantScan(120, 3, 64, 16, dtype=F32, save=True)
        size = plan.workspace.numel()
        plan.workspace = torch.full((size + 4096,), 99, dtype=torch.uint8, device=DEV)[:size]
        forward(cu, d, plan=plan, y=guard[1])
        backward(plan, cu, d)
        assert (guard[0] == 7).all() and (guard[2] == 7).all()
        assert (plan.workspace.as_strided((4096,), (1,), size) == 99).all()


def test_captured_training_step():
    """Forward and backward in one graph, replayed with eager work between, each with a plan of its own."""
    cu = [0, 50, 180]
    x = make(cu, 180, 96, 16, 1, BF16, seed=46)
    d = dev(x)
    s = {m: None if t is None else t.clone() for m, t in d.items()}
    where = offsets(cu)
    plan = lq.LeapQuantScan(180, 2, 96, 16, dtype=BF16, save=True)
    y, S = torch.empty_like(s["x"]), torch.empty_like(s["S0"])
    out = {m: torch.empty_like(s[m]) for m in ("x", "dt", "A", "B", "C", "D", "bias", "z", "S0")}

    def step():
        lq.leapquant_scan_forward(plan, where, s["x"], s["dt"], s["A"], s["B"], s["C"], y, S0=s["S0"], S=S, **weights(s))
        lq.leapquant_scan_backward(plan, where, s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], out["x"], out["dt"],
                                   out["A"], out["B"], out["C"], dD=out["D"], ddt_bias=out["bias"], dz=out["z"], dS=s["dS"],
                                   dS0=out["S0"], **weights(s))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for k in range(4):
        s["x"].copy_((d["x"] * (k + 1)).to(BF16))
        graph.replay()
        p, y2, S2 = forward(cu, s, save=True)
        g2 = backward(p, cu, s)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(S, S2)
        for m in out:
            assert torch.equal(out[m], g2[m]), m


def test_two_streams_at_once():
    """Two calls with a plan each on two streams."""
    cu = [0, 300, 700]
    a, b = (dev(make(cu, 700, 512, 16, 1, BF16, seed=47 + k)) for k in range(2))
    refs = [forward(cu, v)[1:] for v in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for st, v in zip(streams, (a, b)):
        with torch.cuda.stream(st):
            got.append(forward(cu, v)[1:])
    torch.cuda.synchronize()
    for r, g in zip(refs, got):
        assert torch.equal(r[0], g[0]) and torch.equal(r[1], g[1])


def test_refusals_on_the_device():
    d = dev(make([0, 4, 10], 10, 32, 8, 2, F32, seed=48))
    plan = lq.LeapQuantScan(10, 2, 32, 8, groups=2, dtype=F32)
    ok = dict(cu_seqlens=offsets([0, 4, 10]), x=d["x"], dt=d["dt"], A=d["A"], B=d["B"], C=d["C"], y=torch.empty_like(d["x"]))
    lq.leapquant_scan_forward(plan, **ok)
    z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    bad = [dict(cu_seqlens=ok["cu_seqlens"].long()), dict(cu_seqlens=ok["cu_seqlens"].cpu()), dict(A=z(32, 16)),
           dict(A=d["A"].double()), dict(B=z(10, 1, 8)), dict(B=d["B"].half()), dict(C=z(9, 2, 8)), dict(x=z(10, 33)),
           dict(x=z(10, 32).half()), dict(x=z(32, 10).t()), dict(y=z(10, 32).cpu()), dict(D=z(16)), dict(z=z(10, 31)),
           dict(S0=z(1, 32, 8)), dict(S=z(2, 32, 8).double()), dict(x=z(11, 32)), dict(B=z(10, 8, 2).transpose(1, 2))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            lq.leapquant_scan_forward(plan, **{**ok, **kw})
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_scan_forward(plan, **{**ok, "y": d["x"]})
    S = z(2 * 32 * 8 + 8)
    with pytest.raises(lq.LeapQuantError):   # states that overlap in part
        lq.leapquant_scan_forward(plan, **ok, S0=S[:512].view(2, 32, 8), S=S[8:].view(2, 32, 8))


@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_last_input_that_is_not_finite(value, N):
    """It enters the results where the formula has it, and the gradient of A not at all: a step decays the state before
    it.  The sequences end 1, 2, 3 and 4 tokens into a run of the gradient's."""
    cu, c = [0, 5, 11, 18, 26], 70
    x = make(cu, 26, c, N, 1, F32, seed=60 + N)
    for end in cu[1:]:
        x["x"][end - 1, [3, 69]] = value
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    ref, top = reference(cu, x)
    got = backward(plan, cu, d)
    assert torch.isfinite(ref["A"]).all() and torch.isfinite(got["A"]).all()
    check(got["A"], ref["A"], 9 * 8 + 2 * N + c + 160 + 26, "dA", top["A"])
    for t, r in ((y, ref["y"]), (S, ref["S"]), (got["x"], ref["x"]), (got["dt"], ref["dt"]), (got["z"], ref["z"]),
                 (got["B"], ref["B"]), (got["C"], ref["C"]), (got["S0"], ref["S0"]), (got["bias"], ref["bias"])):
        assert torch.equal(torch.isfinite(t.cpu()), torch.isfinite(r))


def test_many_waves_of_a_group():
    """Sums of B's and C's gradients over channels of several waves and groups, the last wave partly full."""
    cu = [0, 37, 90]
    x = make(cu, 90, 2 * 333, 16, 2, F32, seed=70)
    d = dev(x)
    plan, y, S = forward(cu, d, save=True)
    check_all(cu, d, x, y, S, backward(plan, cu, d))


@pytest.mark.parametrize("tokens", [1, 7, 8, 9, 15, 16, 17, 23, 25, 31, 32, 33, 39, 41, 63, 65, 100, 129, 200])
def test_lengths_around_the_chunks(tokens):
    """One sequence of every form: in one chunk, in chunks of a few tokens, in longer ones."""
    x = make([0, tokens], tokens, 72, 16, 1, F32, seed=80 + tokens, slow=-1.0)
    d = dev(x)
    plan, y, S = forward([0, tokens], d, save=True)
    check_all([0, tokens], d, x, y, S, backward(plan, [0, tokens], d))
    y2, S2 = forward([0, tokens], d)[1:]
    assert torch.equal(y, y2) and torch.equal(S, S2)
