"""Plain 64-bit forms of the sequence operators (test infrastructure).

`recurrence` is the definition, token by token, in torch float64; gradients
come from its automatic differentiation, which tests/test_sequence_reference.py
checks against differences.  `head_norm` likewise.

Error bounds (`bound`).  Kernels hold sums, states and statistics in fp32, so
a result is off by accumulated fp32 roundings of relative size U = 2^-24, plus
half a step of its own type.  Along the longest chain of a forward result
stand three sums (with the state: 128 terms; inside a chunk: 64; the
triangular solve: 64) and, for each earlier token, the three roundings of its
update of the state (unit-norm keys and beta <= 1 make the transition
non-expansive, so those add up and do not grow): n = 256 + 3 T roundings.  A
gradient's chain holds a forward chain, the reverse one with five sums for
three, and its own last sum of up to 128: n = 3 * 256 + 6 T.  Each rounding is
relative to the sum's terms, not to its result; the terms are bounded through
the largest entry of the tensor the result belongs to (of a gradient: and of
the sums of the absolute terms, `mag`, where a caller gives them).
"""
import torch

D = 128
U = 2.0 ** -24


def recurrence(cu, q, k, v, beta, alpha, S0, delta=True):
    """cu: list of offsets; all tensors float64 (alpha [T, hv] or [T, hv, 128]).
    Returns o [T, hv, 128] (zeros outside the sequences) and S."""
    T, hv = v.shape[:2]
    group = hv // q.shape[1] if q.shape[1] else 1
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    if alpha.dim() == 2:
        alpha = alpha[..., None]
    out = [torch.zeros_like(v[0]) for _ in range(T)]
    states = []
    for i in range(len(cu) - 1):
        S = S0[i * hv:(i + 1) * hv]
        for t in range(cu[i], cu[i + 1]):
            DS = alpha[t][..., None] * S
            u = v[t] - (DS * k[t][..., None]).sum(1) if delta else v[t]
            S = DS + (beta[t][:, None] * k[t])[..., None] * u[:, None, :]
            out[t] = (S * q[t][..., None]).sum(1)
        states.append(S)
    return (torch.stack(out) if T else v.clone()), torch.cat(states)


def rotate(x, positions, inv_freq, interleaved):
    rot = 2 * inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq
    cos, sin = a.cos(), a.sin()
    z, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((z, rest), -1)


def head_norm(x, kind, eps, weight, scale, positions, inv_freq, interleaved):
    n = 1 if kind == "l2" else D
    y = x / (x.square().sum(-1, keepdim=True) / n + eps).sqrt()
    if weight is not None:
        y = y * weight
    if inv_freq is not None and inv_freq.numel():
        y = rotate(y, positions, inv_freq, interleaved)
    return y * scale


def step(dtype):
    """Half a step of the type, relative."""
    return torch.finfo(dtype).eps / 2


def bound(ref, dtype, n, mag=None):
    """How far each entry of a result may be from `ref` (see the top)."""
    top = (ref.abs() if mag is None else torch.maximum(ref.abs(), mag)).max() if ref.numel() else 0.0
    own = ref.abs() * step(dtype) if dtype != torch.float32 else 0.0
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # results below the type's normal range
    return own + n * U * top * (1 + step(dtype)) + tiny


def check(got, ref, n, name, mag=None):
    dtype = got.dtype
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, name
    assert torch.isfinite(got).all(), f"{name}: not finite"
    off = (got - ref).abs()
    lim = bound(ref, dtype, n, None if mag is None else mag.detach().double().cpu())
    bad = off > lim
    if bad.any():
        worst = int((off - lim).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst by {off.flatten()[worst]:.3e} at "
                             f"{worst} (ref {ref.flatten()[worst]:.3e}, allowed {(torch.zeros_like(off) + lim).flatten()[worst]:.3e})")
