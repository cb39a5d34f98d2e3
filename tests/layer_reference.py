"""Plain 64-bit forms of the operators around the recurrence (test
infrastructure): the short convolution, the selective scan, the block norm, by
their definitions, token by token.  Gradients come from automatic
differentiation, which tests/test_layer_reference.py checks against differences
and, for the scan, against its adjoint written out.

Error bounds (sequence_reference.bound): an entry is off by at most half a step
of its type and n roundings of 2^-24 of the largest sum of absolute terms
(`mag`) of its tensor.

Convolution.  v: width <= 4 products and a bias, 5 roundings.  The activation
adds an exponential (the argument's product, its rest, the instruction, the last
product: 4), a sum, a reciprocal and a product: n = 16 covers them, as the slope
of v silu'(v) is at most 1.1 times its value's.  Gradients: act' has slope at most
1/2, so v's 5 roundings of up to mag_v turn into 3 mag_v of act'; with mag_v <= 16
and the gradient's own 4 + 8 roundings n = 64.  dw, dbias: and one for each token.

Scan.  A step d stands behind 16 roundings (softplus: exponential, quotient,
eight terms, a sum), a decay a = e^(dA) behind those times |dA| and 3 more, a
token's update of the state behind 3.  What token s gives to the state at t has
passed k = t - s decays: 3 k roundings, and 16 k |dA| e^(-k |dA|) <= 16 / e of the
exponents; joined over chunks the exponents are sums of up to k steps, again
at most k / e roundings.  So n = 4 T + 32 of the sums of absolute terms for S, and
with the sum over N states, the skip, the gate n = 4 T + N + 64 for y.  A gradient
joins a state and a gradient of a state (8 T) with sums over states (N) or
channels (`per`) or tokens (T): n = 9 T + 2 N + per + 160.

Block norm.  Each sum of `dim` squares or products and its root: dim / 2 + 4
roundings; activation 8; with two norms n = 2 dim + 64 forward, 4 dim + 128 for
gradients, and one for each row in the weights'.
"""
import torch


def conv(cu, x, w, bias, X0, silu):
    """x [T, c], w [c, K], X0 [seqs, K - 1, c] (float64).  y (zeros outside the
    sequences), X, and v's sums of absolute terms."""
    T, c = x.shape
    K = w.shape[1]
    y = [0 * w[:, 0] for _ in range(T)]  # (part of the graph, also where no sequence has a token)
    mag = [torch.zeros_like(w[:, 0]) for _ in range(T)]
    last = []
    for i in range(len(cu) - 1):
        row = list(X0[i]) + [x[t] for t in range(cu[i], cu[i + 1])]
        for t in range(cu[i], cu[i + 1]):
            p = t - cu[i]
            terms = [row[p + j] * w[:, j] for j in range(K)]
            v = sum(terms) + (0 if bias is None else bias)
            mag[t] = sum(m.abs() for m in terms) + (0 if bias is None else bias.abs())
            y[t] = v * torch.sigmoid(v) if silu else v
        last.append(torch.stack(row[len(row) - (K - 1):]))
    stack = lambda v: torch.stack(v) if T else x.clone()  # noqa: E731
    return stack(y), torch.stack(last), stack(mag)


def step(v, softplus):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())) if softplus else v


def scan(cu, x, dt, A, B, C, D, bias, z, S0, softplus=True):
    """x, dt, z [T, c], A [c, N], B, C [T, G, N], S0 [seqs, c, N] (float64).
    y (zeros outside the sequences) and S."""
    T, c = x.shape
    per = c // B.shape[1]
    y = [torch.zeros_like(A[:, 0]) for _ in range(T)]
    states = []
    for i in range(len(cu) - 1):
        h = S0[i]
        for t in range(cu[i], cu[i + 1]):
            d = step(dt[t] + (0 if bias is None else bias), softplus)
            b, cc = (m[t].repeat_interleave(per, 0) for m in (B, C))
            h = torch.exp(d[:, None] * A) * h + (d * x[t])[:, None] * b
            p = (h * cc).sum(1) + (0 if D is None else D * x[t])
            y[t] = p if z is None else p * z[t] * torch.sigmoid(z[t])
        states.append(h)
    return (torch.stack(y) if T else x.clone()), torch.stack(states)


def scan_adjoint(cu, x, dt, A, B, C, D, bias, z, S0, dy, dS, softplus=True, absolute=False):
    """The gradients by their formulas, and y and S.  absolute: with the absolute
    value of every term instead, the sums that roundings are relative to."""
    f = torch.abs if absolute else lambda v: v  # noqa: E731
    T, c = x.shape
    G, N = B.shape[1:]
    per = c // G
    x, B, C, S0, dS = f(x), f(B), f(C), f(S0), f(dS)
    D = None if D is None else f(D)
    v = dt + (0 if bias is None else bias)
    d = step(v, softplus)
    slope = torch.sigmoid(v) if softplus else torch.ones_like(v)
    gate = torch.ones_like(x) if z is None else f(z * torch.sigmoid(z))
    dp_all = f(dy) * gate
    r = {m: torch.zeros_like(t) for m, t in (("x", x), ("dt", x), ("B", B), ("C", C), ("A", A), ("y", x))}
    r |= {"D": torch.zeros(c).double(), "bias": torch.zeros(c).double(), "S0": dS.clone(), "S": S0.clone()}
    if z is not None:
        r["z"] = torch.zeros_like(x)
        s = torch.sigmoid(z)
        gate_slope = f(s * (1 + z * (1 - s)))
    wide = lambda m: m.repeat_interleave(per, 0)  # noqa: E731
    share = lambda m: m.unflatten(0, (G, per)).sum(1)  # noqa: E731
    for i in range(len(cu) - 1):
        h, before = S0[i], []
        for t in range(cu[i], cu[i + 1]):
            before.append(h)
            h = torch.exp(d[t][:, None] * A) * h + (f(d[t]) * x[t])[:, None] * wide(B[t])
            p = (h * wide(C[t])).sum(1) + (0 if D is None else D * x[t])
            r["y"][t] = p * gate[t]
            if z is not None:
                r["z"][t] = f(dy)[t] * p * gate_slope[t]
        r["S"][i] = h
        g = dS[i]
        for t in reversed(range(cu[i], cu[i + 1])):
            dp, h = dp_all[t], before.pop()
            a, b, cc = torch.exp(d[t][:, None] * A), wide(B[t]), wide(C[t])
            after = a * h + (f(d[t]) * x[t])[:, None] * b
            g = g + cc * dp[:, None]
            e, gb = g * a * h, (g * b).sum(1)
            r["C"][t] = share(after * dp[:, None])
            r["B"][t] = share(g * (f(d[t]) * x[t])[:, None])
            r["A"] += e * f(d[t])[:, None]
            r["x"][t] = gb * f(d[t]) + (0 if D is None else D * dp)
            r["dt"][t] = ((e * f(A)).sum(1) + gb * x[t]) * slope[t]
            r["D"] += dp * x[t]
            r["bias"] += r["dt"][t]
            g = g * a
        r["S0"][i] = g
    return r


def block_norm(a, z, res, gate, scale, out_norm, wo, wi, eps):
    """h and y (float64)."""
    unit = lambda t: t / (t.square().mean(-1, keepdim=True) + eps).sqrt()  # noqa: E731
    n = unit(a) if out_norm else a
    if out_norm and wo is not None:
        n = n * wo
    if z is not None:
        n = n * torch.sigmoid(z) * (z if gate == "silu" else 1)
    h = scale * n + (0 if res is None else res)
    y = unit(h)
    return h, y if wi is None else y * wi
