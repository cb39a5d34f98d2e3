"""What is measured of the operators around the recurrence of a linear-attention
or state space layer: the short causal convolution (whole sequences, single
tokens, training), the selective state space scan (whole sequences, single
tokens, training) and the norms before and after a block with its gate and
residual scale (forward, training).

Layouts: tokens of all sequences behind one another, sequence b holding tokens
cu[b] .. cu[b+1]-1.  Convolution: x, y [tokens, channels], weight [channels,
width], the inputs before a sequence's first token [sequences, width - 1,
channels].  Scan: x, dt, z, y [tokens, channels], A [channels, states], B, C
[tokens, groups, states], states [sequences, channels, states], fp32; channel
c uses group c // (channels / groups).  Norms: a, z, y and the residual stream
[tokens, heads, dim].
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-5


# ---------------------------------------------------------------- the cases
def _conv(name, op, tokens, seqs, channels, dtype, width=4, bias=True, silu=True, state=True, slots=0):
    return {"name": name, "op": op, "tokens": tokens, "seqs": seqs, "channels": channels, "dtype": dtype, "width": width,
            "bias": bias, "silu": silu, "state": state, "slots": slots}


def _scan(name, op, tokens, seqs, channels, dtype, states=16, groups=1, gate=True, state=True, slots=0):
    return {"name": name, "op": op, "tokens": tokens, "seqs": seqs, "channels": channels, "dtype": dtype,
            "states": states, "groups": groups, "gate": gate, "state": state, "slots": slots}


def _norm(name, op, tokens, heads, dim, dtype, stream, out_norm, gate, residual, scale=1.0):
    """stream: the type of the residual stream.  With a residual the stream and its norm are the outputs, without one
    the gated values alone."""
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "dim": dim, "dtype": dtype, "stream": stream,
            "out_norm": out_norm, "gate": gate, "residual": residual, "scale": scale}


def listed():
    return [
        # the next token of 64 running sequences: queries, keys and values of 32 + 32 heads in one convolution
        _conv("conv_step", "conv_step", 64, 0, 8192, "bf16", slots=80),
        # a batch of prompts of mixed lengths through the same layer
        _conv("conv_prompts", "conv", 16384, 24, 8192, "bf16"),
        # a training step of the 16-head layer: its queries, keys and values
        _conv("conv_train", "conv_train", 8192, 4, 6144, "bf16", state=False),
        # the next token of 256 running sequences, a layer of 4,096 channels
        _scan("scan_step", "scan_step", 256, 0, 4096, "bf16", slots=320),
        # one prompt: few channels to fill the chip with, a long recurrence
        _scan("scan_prompt", "scan", 4096, 1, 4096, "bf16", state=False),
        # a batch of prompts of mixed lengths, in half precision
        _scan("scan_ragged", "scan", 16384, 24, 4096, "fp16"),
        # a small training step in full precision, an odd number of channels
        _scan("scan_train_odd", "scan_train", 1021, 3, 1111, "fp32", states=8, gate=False),
        # a training step of a layer of 2,048 channels
        _scan("scan_train", "scan_train", 8192, 4, 2048, "bf16", state=False),
        # the next token of 64 running sequences: outputs of 32 heads, normed and gated
        _norm("norm_step", "norm", 64, 32, 128, "bf16", "bf16", True, "silu", False),
        # the prompts' outputs, normed and gated
        _norm("norm_gate", "norm", 16384, 32, 128, "bf16", "bf16", True, "silu", False),
        # an odd number of rows of an odd width: a scaled block joins the stream, and the stream's norm
        _norm("norm_train_odd", "norm_train", 1021, 1, 1000, "fp32", "fp32", False, "none", True, 0.22),
        # a training step: a block's output normed, gated and joined to a stream in full precision, and its norm
        _norm("norm_train", "norm_train", 8192, 1, 4096, "bf16", "fp32", True, "sigmoid", True, 0.5),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd ones among them."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("conv_step", "conv", "conv_train", "scan_step", "scan", "scan", "scan_train", "norm", "norm_train"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("norm", "norm_train"):
        residual = rng.random() < 0.5
        heads = 1 if residual else rng.choice((4, 8, 16, 32))
        dim = 8 * _between(rng, 8, 1024) if residual else rng.choice((64, 128, 256))
        stream = rng.choice((dtype, "fp32")) if residual else dtype
        c = _norm("", op, _between(rng, 1, min(16384, (1 << 25) // (heads * dim))), heads, dim, dtype, stream,
                  rng.random() < 0.5 or not residual, rng.choice(("none", "silu", "sigmoid")) if residual else "silu",
                  residual, rng.choice((1.0, 0.5, 0.22)) if residual else 1.0)
    elif op in ("conv_step", "scan_step"):
        rows = _between(rng, 1, 256)
        slots = rows + rng.choice((0, 1, 64))
        if op == "conv_step":
            c = _conv("", op, rows, 0, _between(rng, 256, 8192), dtype, rng.choice((2, 3, 4, 4)), rng.random() < 0.5,
                      rng.random() < 0.8, True, slots)
        else:
            groups = rng.choice((1, 1, 2, 4))
            c = _scan("", op, rows, 0, groups * _between(rng, 64, 1024), dtype, rng.choice((8, 16, 16, 32)), groups,
                      rng.random() < 0.7, True, slots)
    elif op in ("conv", "conv_train"):
        channels = _between(rng, 256, 8192)
        tokens = _between(rng, 1, min(16384 if op == "conv" else 8192, (1 << (27 if op == "conv" else 25)) // channels))
        c = _conv("", op, tokens, _between(rng, 1, min(64, tokens)), channels, dtype, rng.choice((2, 3, 4, 4)),
                  rng.random() < 0.5, rng.random() < 0.8, rng.random() < 0.7)
    else:
        groups = rng.choice((1, 1, 2, 4))
        channels, states = groups * _between(rng, 64, 1024), rng.choice((8, 16, 16, 32))
        most = (1 << (29 if op == "scan" else 27)) // (channels * states)
        tokens = _between(rng, 1, min(16384 if op == "scan" else 8192, most))
        c = _scan("", op, tokens, _between(rng, 1, min(64, tokens)), channels, dtype, states, groups, rng.random() < 0.7,
                  rng.random() < 0.7)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: mixed, some of them short or empty, the same ones for every seed."""
    tokens, seqs = case["tokens"], case["seqs"]
    rng = random.Random(7919 * tokens + seqs)
    w = [rng.expovariate(1.0) for _ in range(seqs)]
    cuts = sorted(int(round(tokens * sum(w[:i]) / sum(w))) for i in range(1, seqs))
    ends = [0, *cuts, tokens]
    return [b - a for a, b in zip(ends, ends[1:])]


def _inputs(case, seed):
    """The inputs, from the seed alone, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    op, T, dt = case["op"], case["tokens"], TYPES[case["dtype"]]
    if op in ("norm", "norm_train"):
        heads, dim, stream = case["heads"], case["dim"], TYPES[case["stream"]]
        x = {"a": randn(T, heads, dim).to(dt)}
        # the gate as a fused projection leaves it: a slice of its rows
        x["z"] = randn(T, 2 * heads, dim).to(dt)[:, heads:] if case["gate"] != "none" else None
        x["res"] = (2 * randn(T, heads, dim)).to(stream) if case["residual"] else None
        x["wo"] = 1 + 0.1 * randn(dim) if case["out_norm"] else None
        x["wi"] = 1 + 0.1 * randn(dim) if case["residual"] else None
        if op == "norm_train":
            x["dh"] = randn(T, heads, dim).to(stream)
            x["dy"] = randn(T, heads, dim).to(dt) if case["residual"] else None
        return x
    D, slots = case["channels"], case["slots"]
    x = {}
    if slots:  # running sequences: each row's slot, in any order
        x["slots"] = torch.randperm(slots, generator=g, device="cuda")[:T].to(torch.int32)
    n = slots or case["seqs"]
    if op in ("conv", "conv_step", "conv_train"):
        K = case["width"]
        # what is convolved as a fused projection leaves it: a slice of its rows
        x["x"] = randn(T, D + 64).to(dt)[:, 64:]
        x["w"] = randn(D, K) * K ** -0.5
        x["bias"] = 0.1 * randn(D) if case["bias"] else None
        x["X0"] = randn(n, K - 1, D).to(dt) if case["state"] else None
        if op == "conv_train":
            x["dy"] = randn(T, D).to(dt)
            x["dX"] = randn(n, K - 1, D).to(dt) if case["state"] else None
        return x
    N, G = case["states"], case["groups"]
    # values and gate out of one projection, B and C out of another, beside the 64 values that dt comes from
    rows, low = randn(T, 2 * D).to(dt), randn(T, 64 + 2 * G * N).to(dt)
    x["x"], x["z"] = rows[:, :D], rows[:, D:] if case["gate"] else None
    x["B"], x["C"] = low[:, 64:64 + G * N].unflatten(1, (G, N)), low[:, 64 + G * N:].unflatten(1, (G, N))
    # steps of 0.001 to 0.1, spread over their logarithm, moved by each token; decays 1 .. N as such layers begin with
    x["dt"] = (0.5 * randn(T, D)).to(dt)
    x["dt_bias"] = torch.expm1(torch.exp(math.log(1e-3) + rand(D).double() * math.log(100.0))).log().float()
    x["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * randn(D, N))
    x["D"] = 1 + 0.1 * randn(D)
    x["S0"] = randn(n, D, N) if case["state"] else None
    if op == "scan_train":
        x["dy"] = randn(T, D).to(dt)
        x["dS"] = randn(n, D, N) if case["state"] else None
    return x


def prepare(case, seed):
    s = {"case": dict(case), **_inputs(case, seed)}
    op, T, dt = case["op"], case["tokens"], TYPES[case["dtype"]]
    like = lambda *names: {"d" + m: torch.empty(s[m].shape, dtype=s[m].dtype, device="cuda") for m in names  # noqa: E731
                           if s[m] is not None}
    if own:
        import recurrent_state_quant_amd as lq
    if op in ("norm", "norm_train"):
        s["h"] = torch.empty(s["a"].shape, dtype=TYPES[case["stream"]], device="cuda")
        s["y"] = torch.empty(s["a"].shape, dtype=dt, device="cuda") if case["residual"] else None
        if op == "norm_train":
            s["grads"] = like("a", "z", "res", "wo", "wi")
            if own:
                s["workspace"] = lq.leapquant_block_norm_workspace(T, case["heads"], case["dim"], "cuda")
        return s
    D = case["channels"]
    s["y"] = torch.empty((T, D), dtype=dt, device="cuda")
    if case["slots"]:
        s["S"] = torch.empty_like(s["X0"] if op == "conv_step" else s["S0"]).zero_()  # the states after the token
        return s
    lengths = _lengths(case)
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32)
    s["lengths"], s["cu"] = lengths, cu.cuda()
    if op in ("conv", "conv_train"):
        s["X"] = torch.empty((case["seqs"], case["width"] - 1, D), dtype=dt, device="cuda")
        if op == "conv_train":
            s["grads"] = like("x", "w", "bias", "X0")
            if own:
                s["workspace"] = lq.leapquant_conv_workspace(T, case["seqs"], D, case["width"], "cuda")
        return s
    s["S"] = torch.empty((case["seqs"], D, case["states"]), device="cuda")
    if op == "scan_train":
        s["grads"] = like("x", "dt", "A", "B", "C", "D", "dt_bias", "z", "S0")
    if own:
        s["plan"] = lq.LeapQuantScan(T, case["seqs"], D, case["states"], groups=case["groups"], dtype=dt, device="cuda",
                                     save=op == "scan_train")
    return s


# ---------------------------------------------------------------- the plain forms
def _places(s):
    """Of each token: its sequence and its place in it; and the tokens' number of each sequence."""
    lens = torch.tensor(s["lengths"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
    return seq, torch.arange(len(seq), device="cuda") - (lens.cumsum(0) - lens)[seq], lens


def _act(x, kind):
    return x * torch.sigmoid(x) if kind == "silu" else torch.sigmoid(x)


def _plain_conv(s, x, w, bias, X0):
    """The outputs and the last inputs of every sequence: products with the inputs of each distance, summed."""
    c = s["case"]
    K, D = c["width"], c["channels"]
    if X0 is None:
        X0 = torch.zeros((c["slots"] or c["seqs"], K - 1, D), device="cuda")
    if c["slots"]:
        window = torch.cat((X0[s["slots"].long()], x[:, None]), 1)
        y = (window * w.t()).sum(1)
        last = window[:, 1:]
    else:
        # every sequence behind its earlier inputs, in one row of inputs
        seq, place, lens = _places(s)
        order = torch.arange(c["seqs"], device="cuda")
        first = lens.cumsum(0) - lens + order * (K - 1)
        at = first[seq] + place + K - 1
        before = (first[:, None] + torch.arange(K - 1, device="cuda")).flatten()
        row = torch.zeros((len(at) + len(before), D), device="cuda")
        row = row.index_copy(0, torch.cat((at, before)), torch.cat((x, X0.flatten(0, 1))))
        y = sum(row[at - (K - 1) + j] * w[:, j] for j in range(K))
        last = row[(first + lens)[:, None] + torch.arange(K - 1, device="cuda")]
    if bias is not None:
        y = y + bias
    return (_act(y, "silu") if c["silu"] else y), last


def _doubling(a, b, steps):
    """h_t = a_t h_{t-1} + b_t along the first axis, from zero: runs of 1, 2, 4 .. joined."""
    n = 1
    while n < steps:
        b = torch.cat((b[:n], torch.addcmul(b[n:], a[n:], b[:-n])))
        a = torch.cat((a[:n], a[n:] * a[:-n]))
        n *= 2
    return b


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(s):
    c = s["case"]
    D, N, train = c["channels"], c["states"], c["op"] == "scan_train"
    f = lambda m: None if s.get(m) is None else s[m].float()  # noqa: E731
    x, z, S0, skip = f("x"), f("z"), f("S0"), s["D"]
    Bt, Ct = (f(m).repeat_interleave(D // c["groups"], 1) for m in ("B", "C"))  # [tokens, channels, states]
    v = f("dt") + s["dt_bias"]
    step = _softplus(v)
    a = torch.exp(step[..., None] * s["A"])
    b = (step * x)[..., None] * Bt
    if S0 is None:
        S0 = torch.zeros((c["slots"] or c["seqs"], D, N), device="cuda")
    if c["slots"]:
        h = a * S0[s["slots"].long()] + b
    else:
        seq, place, lens = _places(s)
        head, last = place == 0, place == lens[seq] - 1
        start = torch.where(head[:, None, None], a * S0[seq], 0.0)
        reset = torch.where(head[:, None, None], 0.0, a)
        h = _doubling(reset, b + start, max(s["lengths"]))
        del start, reset
    p = (h * Ct).sum(-1) + skip * x
    out = {"y": (p if z is None else p * _act(z, "silu")).to(s["x"].dtype)}
    if c["slots"]:
        return out, h
    S = S0.clone()
    S[seq[last]] = h[last]
    out["S"] = S
    if not train:
        return out, None
    dy = f("dy")
    dp = dy if z is None else dy * _act(z, "silu")
    end = Ct * dp[..., None]
    if s["dS"] is not None:
        end = end + torch.where(last[:, None, None], s["dS"][seq], 0.0)
    ahead = torch.where(last[:, None, None], 0.0, torch.cat((a[1:], a[:1])))
    gh = _doubling(ahead.flip(0), end.flip(0), max(s["lengths"])).flip(0)  # the gradient of h
    del ahead, end
    before = torch.where(head[:, None, None], S0[seq], torch.cat((h[:1], h[:-1])))
    through = gh * a * before
    dstep = (through * s["A"]).sum(-1) + (gh * Bt).sum(-1) * x
    dv = dstep * torch.sigmoid(v)
    shared = lambda t: t.unflatten(1, (c["groups"], -1)).sum(2)  # noqa: E731
    g = {"dx": (gh * Bt).sum(-1) * step + skip * dp, "ddt": dv, "dA": (through * step[..., None]).sum(0),
         "dB": shared(gh * (step * x)[..., None]), "dC": shared(h * dp[..., None]), "dD": (dp * x).sum(0),
         "ddt_bias": dv.sum(0)}
    if z is not None:
        sz = torch.sigmoid(z)
        g["dz"] = dy * p * sz * (1 + z * (1 - sz))
    if s["S0"] is not None:
        g["dS0"] = torch.zeros_like(S0) if s["dS"] is None else s["dS"].clone()
        g["dS0"][seq[head]] = (a * gh)[head]
    low = ("dx", "ddt", "dB", "dC", "dz")
    return out | {m: t.to(s["x"].dtype) if m in low else t for m, t in g.items()}, None


def _plain_norm(c, a, z, res, wo, wi):
    unit = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)  # noqa: E731
    u = unit(a) * wo if c["out_norm"] else a
    if z is not None:
        u = u * _act(z, c["gate"])
    h = c["scale"] * u
    if res is None:
        return h, None
    h = res + h
    return h, unit(h) * wi


def _plain(s):
    c = s["case"]
    op, train = c["op"], c["op"] in ("conv_train", "norm_train")
    if op in ("scan", "scan_step", "scan_train"):
        out, rows = _plain_scan(s)
        if c["slots"]:
            s["S"][s["slots"].long()] = rows
            out["S"] = s["S"]
        return out
    names = ("x", "w", "bias", "X0") if "conv" in op else ("a", "z", "res", "wo", "wi")
    leaf = [None if s[m] is None else s[m].detach().float().requires_grad_(train) for m in names]
    if op in ("norm", "norm_train"):
        h, y = _plain_norm(c, *leaf)
        r = {"h": h.detach().to(TYPES[c["stream"]])} | ({} if y is None else {"y": y.detach().to(TYPES[c["dtype"]])})
        outs = [(h, s.get("dh")), (y, s.get("dy"))]
    else:
        y, last = _plain_conv(s, *leaf)
        dt = s["x"].dtype
        r = {"y": y.detach().to(dt)}
        if c["slots"]:
            s["S"][s["slots"].long()] = last.to(dt)
            r["S"] = s["S"]
        else:
            r["X"] = last.detach().to(dt)
        outs = [(y, s.get("dy")), (last, s.get("dX"))]
    if train:
        outs = [(o, g.float()) for o, g in outs if o is not None and g is not None]
        ins = [(m, t) for m, t in zip(names, leaf) if t is not None]
        grads = torch.autograd.grad([o for o, _ in outs], [t for _, t in ins], [g for _, g in outs])
        r |= {"d" + m: g.to(s[m].dtype) for (m, _), g in zip(ins, grads)}
    return r


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return _plain(s)
    import recurrent_state_quant_amd as lq
    c = s["case"]
    op = c["op"]
    if op in ("norm", "norm_train"):
        how = dict(z=s["z"], res=s["res"], gate=c["gate"], scale=c["scale"], out_norm=c["out_norm"], out_weight=s["wo"],
                   in_weight=s["wi"], eps=EPS)
        lq.leapquant_block_norm(s["a"], h=s["h"], y=s["y"], **how)
        r = {"h": s["h"]} | ({} if s["y"] is None else {"y": s["y"]})
        if op == "norm_train":
            d = s["grads"]
            lq.leapquant_block_norm_backward(s["a"], d["da"], dh=s["dh"], dy=s["dy"], dz=d.get("dz"), dres=d.get("dres"),
                                             dout_weight=d.get("dwo"), din_weight=d.get("dwi"), workspace=s["workspace"],
                                             **how)
            r |= d
        return r
    if op in ("conv", "conv_step", "conv_train"):
        how = dict(bias=s["bias"], activation="silu" if c["silu"] else "none")
        if op == "conv_step":
            lq.leapquant_conv_step(s["x"], s["w"], s["y"], s["X0"], X_out=s["S"], slots=s["slots"], **how)
            return {"y": s["y"], "S": s["S"]}
        lq.leapquant_conv_forward(s["cu"], s["x"], s["w"], s["y"], X0=s["X0"], X=s["X"], **how)
        r = {"y": s["y"], "X": s["X"]}
        if op == "conv_train":
            d = s["grads"]
            lq.leapquant_conv_backward(s["cu"], s["x"], s["w"], s["dy"], d["dx"], X0=s["X0"], dweight=d["dw"],
                                       dbias=d.get("dbias"), dX=s["dX"], dX0=d.get("dX0"), workspace=s["workspace"], **how)
            r |= d
        return r
    how = dict(D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
    if op == "scan_step":
        lq.leapquant_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["y"], s["S0"], S_out=s["S"], slots=s["slots"],
                               **how)
        return {"y": s["y"], "S": s["S"]}
    lq.leapquant_scan_forward(s["plan"], s["cu"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["y"], S0=s["S0"], S=s["S"],
                              **how)
    r = {"y": s["y"], "S": s["S"]}
    if op == "scan_train":
        d = s["grads"]
        lq.leapquant_scan_backward(s["plan"], s["cu"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["dy"], d["dx"], d["ddt"],
                                   d["dA"], d["dB"], d["dC"], dD=d["dD"], ddt_bias=d["ddt_bias"], dz=d.get("dz"),
                                   dS=s["dS"], dS0=d.get("dS0"), **how)
        r |= d
    return r


def work(case):
    """Bytes: every input read once, every output written once.  Operations: convolution, two for each weight
    (gradient: four more); scan, for each state of each channel and token the decay's product and exponential, two
    products and two sums for the state and the output's two (gradient: seventeen more); norms, about ten a value
    (gradient: twenty more)."""
    op, T, e = case["op"], case["tokens"], SIZE[case["dtype"]]
    train = op.endswith("_train")
    if "norm" in op:
        n, es, gate, res = case["heads"] * case["dim"], SIZE[case["stream"]], case["gate"] != "none", case["residual"]
        once = e * (1 + gate + res) + es * (1 + res)  # a, z, y; h, res
        if train:
            once += e * (1 + gate + res) + es * (1 + res)  # da, dz, dy; dh, dres
        return {"bytes": T * n * once, "flops": T * n * (30 if train else 10)}
    D = case["channels"]
    seqs = T if case["slots"] else case["seqs"]
    sides = 2 if case["state"] else 1
    if "conv" in op:
        K = case["width"]
        token = (4 if train else 2) * e
        states = seqs * (K - 1) * D * e * (sides + (2 if train and case["state"] else 0))
        return {"bytes": T * D * token + states + D * (K + case["bias"]) * 4 * (1 + train),
                "flops": T * D * K * (6 if train else 2)}
    N, G = case["states"], case["groups"]
    token = e * (D * (3 + case["gate"]) + 2 * G * N)
    states = seqs * D * N * 4 * sides
    if train:
        token += e * (D * (3 + case["gate"]) + 2 * G * N)
        states += seqs * D * N * 4 * 2 if case["state"] else 0
    return {"bytes": T * token + states + D * (N + 2) * 4 * (1 + train), "flops": T * D * N * (25 if train else 8)}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    kind = case["op"].split("_")[0]
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[kind](case, s)


def _bounds(c):
    ends = [0]
    for n in _lengths(c):
        ends.append(ends[-1] + n)
    return list(zip(ends, ends[1:]))


def _exact_conv(c, s):
    """Sequence by sequence, on the sequence behind its earlier inputs."""
    K, D, dt = c["width"], c["channels"], TYPES[c["dtype"]]
    w, bias = s["w"].double(), 0.0 if s["bias"] is None else s["bias"].double()
    out = lambda v: v / (1 + torch.exp(-v)) if c["silu"] else v  # noqa: E731
    if c["slots"]:
        at = s["slots"].long()
        rows = [s["X0"][at, j].double() for j in range(K - 1)] + [s["x"].double()]
        y = bias + 0.0 * rows[0]
        for j in range(K):
            y = y + rows[j] * w[:, j]
        S = torch.zeros_like(s["X0"]).double()
        for j in range(K - 1):
            S[at, j] = rows[j + 1]
        return {"y": out(y), "S": S}
    parts = {m: [] for m in ("y", "X", "dx", "dX0")}
    dw, db = torch.zeros((D, K), dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(_bounds(c)):
        n = hi - lo
        early = torch.zeros((K - 1, D), dtype=torch.float64, device="cuda") if s["X0"] is None else s["X0"][i].double()
        row = torch.cat((early, s["x"][lo:hi].double()))
        v = bias + torch.zeros((n, D), dtype=torch.float64, device="cuda")
        for j in range(K):
            v = v + row[j:j + n] * w[:, j]
        parts["y"].append(out(v))
        parts["X"].append(row[n:][None])
        if c["op"] == "conv_train":
            dv = s["dy"][lo:hi].double()
            if c["silu"]:
                sg = 1 / (1 + torch.exp(-v))
                dv = dv * (sg + v * sg * (1 - sg))
            drow = torch.zeros_like(row)
            if s["dX"] is not None:
                drow[n:] += s["dX"][i].double()
            for j in range(K):
                drow[j:j + n] += dv * w[:, j]
                dw[:, j] += (dv * row[j:j + n]).sum(0)
            db += dv.sum(0)
            parts["dx"].append(drow[K - 1:])
            parts["dX0"].append(drow[None, :K - 1])
    r = {m: torch.cat(parts[m]) for m in ("y", "X")}
    if c["op"] == "conv_train":
        r |= {"dx": torch.cat(parts["dx"]), "dw": dw}
        if s["bias"] is not None:
            r["dbias"] = db
        if s["X0"] is not None:
            r["dX0"] = torch.cat(parts["dX0"])
    return r


def _exact_scan(c, s):
    """Token by token, the sequences beside one another: the recurrence, and for training its adjoint."""
    D, N, G, train = c["channels"], c["states"], c["groups"], c["op"] == "scan_train"
    if c["slots"]:
        lengths, n = [1] * c["tokens"], c["tokens"]
    else:
        lengths, n = _lengths(c), c["seqs"]
    steps = max(max(lengths), 1)
    if steps > 8192 or (train and n * steps * D * N * 8 > 96 << 30):
        return None
    b = torch.tensor([i for i, m in enumerate(lengths) for _ in range(m)], device="cuda")
    t = torch.tensor([j for m in lengths for j in range(m)], device="cuda")

    def spread(v):
        y = torch.zeros((steps, n, *v.shape[1:]), dtype=torch.float64, device="cuda")
        y[t, b] = v.double()
        return y

    v = spread(s["dt"].double() + s["dt_bias"].double())
    on = spread(torch.ones((c["tokens"], 1), device="cuda"))
    u = torch.exp(-v.abs())
    step = (v.clamp(min=0) + torch.log1p(u)) * on  # a step of zero leaves the state as it is: behind a sequence's end
    x, Bt, Ct, A, skip = spread(s["x"]), spread(s["B"]), spread(s["C"]), s["A"].double(), s["D"].double()
    wide = lambda m: m.repeat_interleave(D // G, 1)  # noqa: E731
    if s["S0"] is None:
        h = torch.zeros((n, D, N), dtype=torch.float64, device="cuda")
    else:
        h = s["S0"].double() if not c["slots"] else s["S0"][s["slots"].long()].double()
    p, before = torch.empty_like(x), []
    for i in range(steps):
        if train:
            before.append(h)
        h = torch.exp(step[i][..., None] * A) * h + (step[i] * x[i])[..., None] * wide(Bt[i])
        p[i] = (h * wide(Ct[i])).sum(-1) + skip * x[i]
    if s["z"] is not None:
        z = spread(s["z"])
        sig = 1 / (1 + torch.exp(-z))
        gate = z * sig
    else:
        gate = torch.ones_like(x)
    r = {"y": (p * gate)[t, b]}
    if c["slots"]:
        r["S"] = torch.zeros(s["S0"].shape, dtype=torch.float64, device="cuda")
        r["S"][s["slots"].long()] = h
        return r
    r["S"] = h
    if not train:
        return r
    dy = spread(s["dy"])
    dp = dy * gate
    g = torch.zeros_like(h) if s["dS"] is None else s["dS"].double()
    dx, dstep, dB, dC = (torch.empty_like(m) for m in (x, x, Bt, Ct))
    dA = torch.zeros_like(A)
    share = lambda m: m.unflatten(1, (G, D // G)).sum(2)  # noqa: E731
    after = h
    for i in reversed(range(steps)):
        h = before.pop()
        dC[i] = share(after * dp[i][..., None])
        g = g + dp[i][..., None] * wide(Ct[i])
        d = torch.exp(step[i][..., None] * A)
        by = g * d * h
        gB = (g * wide(Bt[i])).sum(-1)
        dB[i] = share(g * (step[i] * x[i])[..., None])
        dx[i] = gB * step[i] + skip * dp[i]
        dstep[i] = (by * A).sum(-1) + gB * x[i]
        dA += (by * step[i][..., None]).sum(0)
        g = g * d
        after = h
    dv = dstep * torch.where(v >= 0, 1 / (1 + u), u / (1 + u)) * on
    r |= {"dx": dx[t, b], "ddt": dv[t, b], "dA": dA, "dB": dB[t, b], "dC": dC[t, b], "dD": (dp * x * on).sum((0, 1)),
          "ddt_bias": dv.sum((0, 1))}
    if s["z"] is not None:
        r["dz"] = (dy * p * (sig + z * sig * (1 - sig)))[t, b]
    if s["S0"] is not None:
        r["dS0"] = g
    return r


def _exact_norm(c, s):
    dim, scale = c["dim"], c["scale"]
    a = s["a"].double()
    ra = 1 / ((a * a).sum(-1, keepdim=True) / dim + EPS).sqrt()
    wo = s["wo"].double() if c["out_norm"] else None
    n = a * ra * wo if c["out_norm"] else a
    gate = dgate = None
    if s["z"] is not None:
        z = s["z"].double()
        sig = 1 / (1 + torch.exp(-z))
        gate, dgate = (z * sig, sig + z * sig * (1 - sig)) if c["gate"] == "silu" else (sig, sig * (1 - sig))
    u = n if gate is None else n * gate
    h = scale * u if s["res"] is None else s["res"].double() + scale * u
    r = {"h": h}
    if s["res"] is not None:
        rh = 1 / ((h * h).sum(-1, keepdim=True) / dim + EPS).sqrt()
        r["y"] = h * rh * s["wi"].double()
    if c["op"] != "norm_train":
        return r

    def back(x, m, w, g):
        """The gradients of x * m * w, m the reciprocal root mean square of x, from g."""
        gw = g * w
        return m * gw - x * m ** 3 * (x * gw).sum(-1, keepdim=True) / dim, (g * x * m).sum((0, 1))

    dh = s["dh"].double()
    if s["res"] is not None:
        more, r["dwi"] = back(h, rh, s["wi"].double(), s["dy"].double())
        dh = dh + more
        r["dres"] = dh
    du = scale * dh
    if gate is not None:
        r["dz"], du = du * n * dgate, du * gate
    if c["out_norm"]:
        r["da"], r["dwo"] = back(a, ra, wo, du)
    else:
        r["da"] = du
    return r
