"""What is measured of the sequence operators: the gated delta rule over whole
sequences (forward; forward and backward) and the norm of query and key heads
with the position rotation (forward; forward and backward).

Layouts: tokens of all sequences behind one another, sequence b holding tokens
cu[b] .. cu[b+1]-1; q, k [tokens, heads_k, 128], v, o [tokens, heads_v, 128];
beta [tokens, heads_v]; alpha [tokens, heads_v] (gdn) or [tokens, heads_v, 128]
(kda); states [sequences * heads_v, 128, 128], fp32.  Value head h uses query
and key head h // (heads_v / heads_k).
"""
import random

import torch

own = False

D = 128
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---------------------------------------------------------------- the cases
def _sequence(name, op, tokens, seqs, heads_k, heads_v, dtype, gate="gdn", delta=True, shift=4.0, state=True):
    return {"name": name, "op": op, "tokens": tokens, "seqs": seqs, "heads_k": heads_k, "heads_v": heads_v,
            "dtype": dtype, "gate": gate, "delta": delta, "shift": shift, "state": state}


def _norm(name, op, tokens, heads_q, heads_k, dtype, out, kind="l2", weight=False, rot=0, interleaved=False):
    return {"name": name, "op": op, "tokens": tokens, "heads_q": heads_q, "heads_k": heads_k, "dtype": dtype,
            "out": out, "kind": kind, "weight": weight, "rot": rot, "interleaved": interleaved}


def listed():
    return [
        # a few tokens for each of 64 running sequences of the 32-head layer: drafted tokens to verify
        _sequence("few_tokens", "prefill", 201, 64, 32, 32, "bf16"),
        # one prompt through the 32-head layer: few heads to fill the chip with, a long scan
        _sequence("prompt_4096", "prefill", 4096, 1, 32, 32, "bf16", state=False),
        # a batch of prompts of mixed lengths, two value heads for each key head
        _sequence("prompts_ragged", "prefill", 16384, 24, 16, 32, "bf16"),
        # a per-channel gate, in full precision, strong decays as in the decode workloads
        _sequence("prompts_kda", "prefill", 3001, 5, 32, 32, "fp32", gate="kda", shift=0.0),
        # a small training step in full precision, strong decays
        _sequence("train_small", "train", 509, 3, 4, 4, "fp32", shift=0.0),
        # a training step of the 16-head layer
        _sequence("train_h16", "train", 8192, 4, 16, 16, "bf16", state=False),
        # a packed batch of documents, four value heads for each key head, in half precision
        _sequence("train_packed", "train", 5000, 19, 4, 16, "fp16"),
        # the next token of 256 running sequences of the 32-head layer, for the fp32 decode call
        _norm("norm_decode", "norm", 256, 32, 32, "bf16", "fp32"),
        # the prompts' queries and keys, half of each head rotated
        _norm("norm_prompts", "norm", 16384, 16, 16, "bf16", "bf16", kind="rms", weight=True, rot=64),
        # an odd number of tokens, all of each head rotated in neighbouring pairs, full precision
        _norm("norm_train_odd", "norm_train", 1021, 16, 4, "fp32", "fp32", rot=128, interleaved=True),
        # the queries and keys of the training step, with learned weights
        _norm("norm_train", "norm_train", 8192, 16, 16, "bf16", "bf16", kind="rms", weight=True, rot=128),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, odd ones among them."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "train", "norm", "norm_train"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("norm", "norm_train"):
        rot = rng.choice((0, 32, 64, 96, 128))
        c = _norm("", op, _between(rng, 1, 16384 if op == "norm" else 8192), rng.choice((4, 8, 16, 32)),
                  rng.choice((1, 2, 4, 8, 16)), dtype, rng.choice((dtype, "fp32")), rng.choice(("l2", "rms")),
                  rng.random() < 0.5, rot, rot > 0 and rng.random() < 0.5)
    else:
        heads_k = rng.choice((1, 2, 4, 8, 16))
        heads_v = min(32, heads_k * rng.choice((1, 1, 2, 4)))
        most = 1 << 18 if op == "prefill" else 1 << 16  # tokens times value heads
        tokens = _between(rng, 1, min(16384 if op == "prefill" else 4096, most // heads_v))
        seqs = _between(rng, 1, min(64, tokens))
        gate = rng.choice(("gdn", "gdn", "kda")) if op == "prefill" else "gdn"
        if gate == "kda":
            tokens = min(tokens, (1 << 17) // heads_v)
        c = _sequence("", op, tokens, min(seqs, tokens), heads_k, heads_v, dtype, gate, rng.random() < 0.8,
                      rng.choice((0.0, 2.0, 4.0)), rng.random() < 0.7)
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
    T, dt = case["tokens"], TYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        hq, hk, out = case["heads_q"], case["heads_k"], TYPES[case["out"]]
        # queries and keys as a fused projection leaves them: slices of its rows
        rows = (randn(T, hq + hk + 2, D) * 3).to(dt)
        x = {"q": rows[:, :hq], "k": rows[:, hq:hq + hk]}
        x["wq"] = 1 + 0.1 * randn(D) if case["weight"] else None
        x["wk"] = 1 + 0.1 * randn(D) if case["weight"] else None
        if case["rot"]:
            half = case["rot"] // 2
            x["pos"] = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda", dtype=torch.int64)
            x["freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        if case["op"] == "norm_train":
            x["dq_out"], x["dk_out"] = randn(T, hq, D).to(out), randn(T, hk, D).to(out)
        return x
    hk, hv = case["heads_k"], case["heads_v"]
    n = case["seqs"] * hv
    unit = lambda t: t / torch.linalg.vector_norm(t, dim=-1, keepdim=True)  # noqa: E731
    x = {"q": (unit(randn(T, hk, D)) * D ** -0.5).to(dt), "k": unit(randn(T, hk, D)).to(dt)}
    # the values as a fused projection leaves them: a slice of its rows
    x["v"] = randn(T, 2 * hk + hv, D)[:, 2 * hk:].to(dt)
    x["beta"] = torch.sigmoid(randn(T, hv))
    shape = (T, hv) if case["gate"] == "gdn" else (T, hv, D)
    x["alpha"] = torch.exp(-torch.nn.functional.softplus(randn(*shape) - case["shift"]))
    x["S0"] = 0.02 * randn(n, D, D) if case["state"] else None
    if case["op"] == "train":
        x["do"] = randn(T, hv, D).to(dt)
        x["dS"] = 0.02 * randn(n, D, D) if case["state"] else None
    return x


def prepare(case, seed):
    s = {"case": dict(case), **_inputs(case, seed)}
    T, dt = case["tokens"], TYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        s["q_out"] = torch.empty((T, case["heads_q"], D), dtype=TYPES[case["out"]], device="cuda")
        s["k_out"] = torch.empty((T, case["heads_k"], D), dtype=TYPES[case["out"]], device="cuda")
        if case["op"] == "norm_train":
            s["dq"] = torch.empty((T, case["heads_q"], D), dtype=dt, device="cuda")
            s["dk"] = torch.empty((T, case["heads_k"], D), dtype=dt, device="cuda")
            s["dwq"] = torch.empty(D, device="cuda") if case["weight"] else None
            s["dwk"] = torch.empty(D, device="cuda") if case["weight"] else None
            if own:
                import recurrent_state_quant_amd as lq
                s["workspace"] = lq.leapquant_head_norm_workspace(T, case["heads_q"], case["heads_k"], "cuda")
        return s
    hk, hv, n = case["heads_k"], case["heads_v"], case["seqs"] * case["heads_v"]
    lengths = _lengths(case)
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32)
    s["lengths"], s["cu"] = lengths, cu.cuda()
    s["o"] = torch.empty((T, hv, D), dtype=dt, device="cuda")
    s["S"] = torch.empty((n, D, D), device="cuda")
    if case["op"] == "train":
        s["dq"], s["dk"] = (torch.empty((T, hk, D), dtype=dt, device="cuda") for _ in range(2))
        s["dv"] = torch.empty((T, hv, D), dtype=dt, device="cuda")
        s["dbeta"], s["dalpha"] = torch.empty_like(s["beta"]), torch.empty_like(s["alpha"])
        s["dS0"] = torch.empty((n, D, D), device="cuda") if case["state"] else None
    if own:
        import recurrent_state_quant_amd as lq
        s["plan"] = lq.LeapQuantSequence(T, case["seqs"], hk, hv, gate=case["gate"], dtype=dt, device="cuda",
                                         flags=0 if case["delta"] else lq.LQ_NO_DELTA, save=case["op"] == "train")
    return s


# ---------------------------------------------------------------- the plain forms
def _padded(x, lengths, chunk, fill=0.0):
    """[tokens, ...] -> [sequences, whole chunks, ...], in fp32, and the tokens' places in it."""
    steps = max(1, -(-max(lengths) // chunk)) * chunk
    lens = torch.tensor(lengths, device=x.device)
    at = torch.repeat_interleave(torch.arange(len(lengths), device=x.device) * steps - (lens.cumsum(0) - lens), lens)
    at = at + torch.arange(x.shape[0], device=x.device)
    y = torch.full((len(lengths) * steps, *x.shape[1:]), fill, device=x.device)
    return y.index_copy(0, at, x.float()).unflatten(0, (len(lengths), steps)), at


def _chunked(x, chunk):
    """[sequences, steps, heads, ...] -> [sequences, heads, chunks, chunk, ...]"""
    return x.unflatten(1, (-1, chunk)).movedim(3, 1)


def _plain_sequence(c, lengths, q, k, v, beta, alpha, S0):
    """Chunks of tokens, the products within all chunks at once, the state from chunk to chunk (a recurrence: one
    loop over the chunks).  Decays are sums of logarithms in 64 bits."""
    C = 64 if c["gate"] == "gdn" else 16
    group = c["heads_v"] // c["heads_k"]
    pad = lambda x, fill=0.0: _padded(x, lengths, C, fill)  # noqa: E731
    (vp, at), (bp, _), (ap, _) = pad(v), pad(beta), pad(alpha, 1.0)
    qp, kp = (pad(x)[0].repeat_interleave(group, 2) for x in (q, k))
    q, k, v, beta, alpha = (_chunked(x, C) for x in (qp, kp, vp, bp, ap))
    i = torch.arange(C, device=q.device)
    low, strict = i[:, None] >= i, i[:, None] > i
    log = alpha.double().log().cumsum(3)
    if c["gate"] == "gdn":
        L = torch.exp((log[..., :, None] - log[..., None, :]).masked_fill(~low, float("-inf"))).float()
        A = k @ k.transpose(-1, -2).contiguous() * L
        P = q @ k.transpose(-1, -2).contiguous() * L
        log = log[..., None]
    else:
        L = torch.exp((log[..., :, None, :] - log[..., None, :, :]).masked_fill(~low[..., None], float("-inf"))).float()
        L = L * k[..., None, :, :]
        A, P = (L * k[..., :, None, :]).sum(-1), (L * q[..., :, None, :]).sum(-1)
    P = P * beta[..., None, :]
    T = torch.eye(C, device=q.device, dtype=torch.float64)
    if c["delta"]:  # the inverse of a unit triangle, as a product: (I - M)(I + M^2)(I + M^4) ...
        M = (A * beta[..., None, :]).masked_fill(~strict, 0.0).double()
        M2 = M @ M
        M4 = M2 @ M2
        M8 = M4 @ M4
        T = (T - M) @ (T + M2) @ (T + M4) @ (T + M8)
        if C == 64:
            M16 = M8 @ M8
            T = T + T @ M16
            T = T + T @ (M16 @ M16)
    T = T.float()
    decay = torch.exp(log).float()
    gk, gq = decay * k, decay * q
    kt = (torch.exp(log[..., -1:, :] - log).float() * beta[..., None] * k).transpose(-1, -2).contiguous()
    last = decay[..., -1, :, None]
    S = torch.zeros((*q.shape[:2], D, D), device=q.device) if S0 is None else S0.view(*q.shape[:2], D, D)
    out = []
    for n in range(q.shape[2]):
        x = v[:, :, n] - gk[:, :, n] @ S if c["delta"] else v[:, :, n]
        u = T[:, :, n] @ x if c["delta"] else x
        out.append(gq[:, :, n] @ S + P[:, :, n] @ u)
        S = last[:, :, n] * S + kt[:, :, n] @ u
    o = torch.stack(out, 2).movedim(1, 3).flatten(0, 2)[at]
    return o, S.flatten(0, 1)


def _plain_norm(c, x, w, scale, pos, freq):
    x = x.float()
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) / (1 if c["kind"] == "l2" else D) + 1e-6)
    y = x * r * scale
    if w is not None:
        y = y * w
    if not c["rot"]:
        return y
    a = pos.double()[:, None, None] * freq
    cos, sin = a.cos().float(), a.sin().float()
    z, rest = y[..., :c["rot"]], y[..., c["rot"]:]
    if c["interleaved"]:
        a, b = z[..., 0::2], z[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)
    a, b = z.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)


def _plain(s):
    c = s["case"]
    train = c["op"] in ("train", "norm_train")
    leaf = lambda t: None if t is None else t.detach().float().requires_grad_(train)  # noqa: E731
    if c["op"] in ("norm", "norm_train"):
        q, k, wq, wk = (leaf(s[x]) for x in ("q", "k", "wq", "wk"))
        pos, freq = s.get("pos"), s.get("freq")
        qo, ko = _plain_norm(c, q, wq, D ** -0.5, pos, freq), _plain_norm(c, k, wk, 1.0, pos, freq)
        out = TYPES[c["out"]]
        r = {"q": qo.detach().to(out), "k": ko.detach().to(out)}
        if train:
            ins = [x for x in (q, k, wq, wk) if x is not None]
            g = torch.autograd.grad((qo, ko), ins, (s["dq_out"].float(), s["dk_out"].float()))
            r |= {"dq": g[0].to(s["q"].dtype), "dk": g[1].to(s["k"].dtype)}
            if wq is not None:
                r |= {"dwq": g[2], "dwk": g[3]}
        return r
    q, k, v, beta, alpha, S0 = (leaf(s[x]) for x in ("q", "k", "v", "beta", "alpha", "S0"))
    o, S = _plain_sequence(c, s["lengths"], q, k, v, beta, alpha, S0)
    dt = s["q"].dtype
    r = {"o": o.detach().to(dt), "S": S.detach()}
    if train:
        ins = [x for x in (q, k, v, beta, alpha, S0) if x is not None]
        outs = (o, S) if s["dS"] is not None else (o,)
        g = torch.autograd.grad(outs, ins, (s["do"].float(), s["dS"])[:len(outs)])
        r |= {"dq": g[0].to(dt), "dk": g[1].to(dt), "dv": g[2].to(dt), "dbeta": g[3], "dalpha": g[4]}
        if S0 is not None:
            r["dS0"] = g[5]
    return r


# ---------------------------------------------------------------- one pass
def run(s):
    if not own:
        return _plain(s)
    import recurrent_state_quant_amd as lq
    c = s["case"]
    if c["op"] in ("norm", "norm_train"):
        how = dict(norm=c["kind"], eps=1e-6, q_weight=s["wq"], k_weight=s["wk"], q_scale=D ** -0.5,
                   positions=s.get("pos"), inv_freq=s.get("freq"), interleaved=c["interleaved"])
        lq.leapquant_head_norm(s["q"], s["k"], s["q_out"], s["k_out"], **how)
        r = {"q": s["q_out"], "k": s["k_out"]}
        if c["op"] == "norm_train":
            lq.leapquant_head_norm_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                            dq_weight=s["dwq"], dk_weight=s["dwk"], workspace=s["workspace"], **how)
            r |= {"dq": s["dq"], "dk": s["dk"]}
            if c["weight"]:
                r |= {"dwq": s["dwq"], "dwk": s["dwk"]}
        return r
    lq.leapquant_sequence_forward(s["plan"], s["cu"], s["q"], s["k"], s["v"], s["beta"], s["alpha"], s["o"],
                                  S0=s["S0"], S=s["S"])
    r = {"o": s["o"], "S": s["S"]}
    if c["op"] == "train":
        lq.leapquant_sequence_backward(s["plan"], s["cu"], s["q"], s["k"], s["beta"], s["alpha"], s["do"], s["dq"],
                                       s["dk"], s["dv"], s["dbeta"], s["dalpha"], dS=s["dS"], dS0=s["dS0"])
        r |= {x: s[x] for x in ("dq", "dk", "dv", "dbeta", "dalpha")}
        if c["state"]:
            r["dS0"] = s["dS0"]
    return r


def work(case):
    """Bytes: every input read once, every output written once.  Operations: forward, the three products of a
    128 x 128 state and a vector for each token and value head (state times key, state times query, update);
    backward, six more (the gradient's two updates and four products)."""
    T, e = case["tokens"], SIZE[case["dtype"]]
    train = case["op"] in ("train", "norm_train")
    if case["op"] in ("norm", "norm_train"):
        heads, out = case["heads_q"] + case["heads_k"], SIZE[case["out"]]
        per = 2 * e + 2 * out if train else e + out
        return {"bytes": T * heads * D * per + (T * 8 if case["rot"] else 0), "flops": T * heads * D * (24 if train else 8)}
    hk, hv, n = case["heads_k"], case["heads_v"], case["seqs"] * case["heads_v"]
    gate = 4 if case["gate"] == "gdn" else 4 * D
    token = 2 * hk * D * e + 2 * hv * D * e + hv * (4 + gate)
    states = (2 if case["state"] else 1) * n * D * D * 4
    if train:
        token += 2 * hk * D * e + 2 * hv * D * e + hv * (4 + gate)
        states += (2 if case["state"] else 0) * n * D * D * 4
    return {"bytes": T * token + states, "flops": T * hv * 2 * D * D * (9 if train else 3)}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_norm(case, s) if case["op"] in ("norm", "norm_train") else _exact_sequence(case, s)


def _exact_sequence(c, s):
    """Token by token: the recurrence, and for training its adjoint."""
    T, hk, hv, B = c["tokens"], c["heads_k"], c["heads_v"], c["seqs"]
    lengths = _lengths(c)
    steps = max(max(lengths), 1)
    train = c["op"] == "train"
    if train and B * steps * hv * D * D * 8 > 96 << 30:
        return None
    b = torch.tensor([i for i, n in enumerate(lengths) for _ in range(n)], device="cuda")
    t = torch.tensor([j for n in lengths for j in range(n)], device="cuda")

    def spread(x, fill=0.0):
        y = torch.full((steps, B, *x.shape[1:]), fill, dtype=torch.float64, device="cuda")
        y[t, b] = x.double()
        return y

    q, k = (spread(s[x]).repeat_interleave(hv // hk, 2) for x in ("q", "k"))
    v, beta, alpha = spread(s["v"]), spread(s["beta"])[..., None], spread(s["alpha"], 1.0)
    if c["gate"] == "gdn":
        alpha = alpha[..., None]
    if s["S0"] is None:
        S = torch.zeros((B, hv, D, D), dtype=torch.float64, device="cuda")
    else:
        S = s["S0"].double().view(B, hv, D, D)
    o, u, before = torch.empty_like(v), torch.empty_like(v), []
    for i in range(steps):
        if train:
            before.append(S)
        bt = alpha[i] * k[i] if c["delta"] else torch.zeros_like(k[i])
        u[i] = v[i] - (S * bt[..., None]).sum(-2)
        S = alpha[i][..., None] * S + (beta[i] * k[i])[..., None] * u[i][..., None, :]
        o[i] = (S * q[i][..., None]).sum(-2)
    r = {"o": o[t, b], "S": S.flatten(0, 1)}
    if not train:
        return r
    do = spread(s["do"])
    G = torch.zeros_like(S) if s["dS"] is None else s["dS"].double().view(B, hv, D, D)
    dq, dk, dv, dbeta, dalpha = (torch.empty_like(x) for x in (q, k, v, beta, alpha))
    after = S
    for i in reversed(range(steps)):
        S = before.pop()
        dq[i] = (after * do[i][..., None, :]).sum(-1)
        G = G + q[i][..., None] * do[i][..., None, :]
        du = (G * (beta[i] * k[i])[..., None]).sum(-2)
        dw = (G * u[i][..., None, :]).sum(-1)
        db = -(S * du[..., None, :]).sum(-1) if c["delta"] else torch.zeros_like(dw)
        dv[i], dk[i] = du, beta[i] * dw + alpha[i] * db
        dbeta[i] = (dw * k[i]).sum(-1, keepdim=True)
        dalpha[i] = ((G * S).sum((-1, -2)) + (db * k[i]).sum(-1))[..., None]
        G = alpha[i][..., None] * G
        if c["delta"]:
            G = G - (alpha[i] * k[i])[..., None] * du[..., None, :]
        after = S
    shared = lambda x: x[t, b].unflatten(1, (hk, hv // hk)).sum(2)  # noqa: E731
    r |= {"dq": shared(dq), "dk": shared(dk), "dv": dv[t, b], "dbeta": dbeta[t, b][..., 0], "dalpha": dalpha[t, b][..., 0]}
    if s["S0"] is not None:
        r["dS0"] = G.flatten(0, 1)
    return r


def _exact_norm(c, s):
    r, n, rot = {}, (1 if c["kind"] == "l2" else D), c["rot"]
    if rot:  # the pairs' first and second places, and the turn as a complex number
        even = torch.arange(rot // 2, device="cuda")
        first, second = (2 * even, 2 * even + 1) if c["interleaved"] else (even, even + rot // 2)
        a = s["pos"].double()[:, None, None] * s["freq"]
        turn = torch.complex(a.cos(), a.sin())

    def turned(y, by):
        y = y.clone()
        if rot:
            z = torch.complex(y[..., first], y[..., second]) * by
            y[..., first], y[..., second] = z.real, z.imag
        return y

    for h, scale in (("q", D ** -0.5), ("k", 1.0)):
        x = s[h].double()
        w = 1.0 if s["w" + h] is None else s["w" + h].double()
        m = 1 / ((x * x).sum(-1, keepdim=True) / n + 1e-6).sqrt()
        r[h] = turned(x * m * w * scale, turn if rot else None)
        if c["op"] == "norm_train":
            g = turned(s["d%s_out" % h].double(), turn.conj() if rot else None) * scale
            r["d" + h] = m * w * g - x * m ** 3 * (x * w * g).sum(-1, keepdim=True) / n
            if c["weight"]:
                r["dw" + h] = (g * x * m).sum((0, 1))
    return r
