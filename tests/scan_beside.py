"""The selective scan and its gradient in 64 bits with the sequences beside one
another, on the device that the inputs are on (test infrastructure): what
layer_reference.scan_adjoint computes one sequence after the other, for sizes at
which that takes too long.  tests/test_layer_rules.py compares the two."""
import torch


def scan_adjoint(cu, x, dt, A, B, C, D, bias, z, S0, dy, dS, softplus=True, absolute=False):
    """Arguments and results of layer_reference.scan_adjoint (float64).  absolute: where its bounds take the largest
    entry of a tensor, these are taken entry by entry, so the slope of the gate s (1 + z (1 - s)), which has a zero at z =
    -1.28, counts by its terms too: 1 - s is off by a rounding of 1, and so the slope by s |z| of them, however near its
    own value is to zero."""
    f = torch.abs if absolute else lambda v: v  # noqa: E731
    T, c = x.shape
    G, N = B.shape[1:]
    lens = [b - a for a, b in zip(cu, cu[1:])]
    steps, n = max(lens + [0]), len(lens)
    place = torch.tensor([t for m in lens for t in range(m)], dtype=torch.long, device=x.device)
    seq = torch.tensor([i for i, m in enumerate(lens) for _ in range(m)], dtype=torch.long, device=x.device)

    def beside(v):
        """[steps, sequences, ..]: zeros behind a sequence's end."""
        y = v.new_zeros((steps, n, *v.shape[1:]))
        y[place, seq] = v[cu[0]:cu[-1]]
        return y

    def behind(v):
        y = v.new_zeros((T, *v.shape[2:]))
        y[cu[0]:cu[-1]] = v[place, seq]
        return y

    on = beside(torch.ones_like(x[:, :1]))
    v = beside(dt + (0 if bias is None else bias))
    u = torch.exp(-v.abs())
    # a step of zero leaves the state as it is: behind a sequence's end
    d = on * (v.clamp(min=0) + torch.log1p(u) if softplus else v)
    slope = torch.where(v >= 0, 1 / (1 + u), u / (1 + u)) if softplus else torch.ones_like(v)
    step, x, B, C, dy, skip = f(d), beside(f(x)), beside(f(B)), beside(f(C)), beside(f(dy)), 0 if D is None else f(D)
    gate = gate_slope = torch.ones_like(x)
    if z is not None:
        z = beside(z)
        s = torch.sigmoid(z)
        gate, gate_slope = f(z * s), s * (1 + f(z) * (1 - s))
    wide = lambda m: m.repeat_interleave(c // G, 1)  # noqa: E731
    share = lambda m: m.unflatten(1, (G, c // G)).sum(2)  # noqa: E731
    h, before, p = f(S0), [], torch.zeros_like(x)
    for t in range(steps):
        before.append(h)
        h = torch.exp(d[t][..., None] * A) * h + (step[t] * x[t])[..., None] * wide(B[t])
        p[t] = (h * wide(C[t])).sum(-1) + skip * x[t]
    dp = dy * gate
    r = {"y": behind(p * gate), "S": h, "A": torch.zeros_like(A), "D": (dp * x).sum((0, 1))}
    if z is not None:
        r["z"] = behind(dy * p * gate_slope)
    g, after = f(dS), h
    dx, ddt, dB, dC = (torch.zeros_like(m) for m in (x, x, B, C))
    for t in reversed(range(steps)):
        h = before.pop()
        dC[t] = share(after * dp[t][..., None])
        g = g + dp[t][..., None] * wide(C[t])
        a = torch.exp(d[t][..., None] * A)
        e, gb = g * a * h, (g * wide(B[t])).sum(-1)
        dB[t] = share(g * (step[t] * x[t])[..., None])
        dx[t] = gb * step[t] + skip * dp[t]
        ddt[t] = ((e * f(A)).sum(-1) + gb * x[t]) * slope[t] * on[t]
        r["A"] += (e * step[t][..., None]).sum(0)
        g, after = g * a, h
    return r | {"x": behind(dx), "dt": behind(ddt), "B": behind(dB), "C": behind(dC), "bias": ddt.sum((0, 1)), "S0": g}
