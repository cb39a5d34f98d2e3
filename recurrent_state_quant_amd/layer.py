"""Python binding of the operators around the recurrence (argument marshalling
only): the short causal convolution, the selective state space scan and the
norms before and after a block.  See include/leapquant.h for the semantics of
each call.
"""
import ctypes

import torch

from . import _lib as L
from .api import _F32, _I32, _ptr
from .sequence import _bytes, _dtype_id, _launch, _rows

_ACTS = {"none": L.LQ_ACT_NONE, None: L.LQ_ACT_NONE, "silu": L.LQ_ACT_SILU, "sigmoid": L.LQ_ACT_SIGMOID}


def _act(kind, names):
    if kind not in names:
        raise ValueError(f"unknown activation {kind!r}")
    return _ACTS[kind]


def _channels(x, dtype, shape, name, device):
    """A strided [tokens, channels] tensor as lq_rows (None as it is)."""
    if x is None:
        return None
    r = _rows(x, dtype, shape, name, device)
    if x.stride(1) != 1 and shape[1] > 1 and x.numel():
        raise ValueError(f"{name}: the channels of a token must be contiguous")
    return r


def _heads(x, dtype, shape, name, device):
    return None if x is None else _rows(x, dtype, shape, name, device)


def _dense(x, dtype, shape, name, device):
    """A contiguous tensor's address (None as it is).  Every check passes at once as a rule (a step of the
    convolution, with five such arguments, 12.4 us on the host, 11.3 so); otherwise _ptr names what is wrong."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device and (
            device.type == "cuda" and x.is_contiguous()):
        return x.data_ptr() or None
    return _ptr(x, dtype, shape, name, device)


def _given(x, dtype, shape, name, device):
    """The same of an argument that has to be given."""
    return _ptr(x, dtype, shape, name, device) if x is None else _dense(x, dtype, shape, name, device)


def _matrix(x, name):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return x


def _offsets(cu, device):
    """(cu_seqlens pointer, sequences) of packed sequences."""
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of sequences + 1 offsets")
    return _dense(cu, _I32, (cu.numel(),), "cu_seqlens", device), cu.numel() - 1


def _space(workspace, device):
    if workspace is None:
        return [None, 0]
    return [_dense(workspace, torch.uint8, (workspace.numel(),), "workspace", device), workspace.numel()]


def _conv_params(x, weight, bias, activation, seqs):
    T, c = _matrix(x, "x").shape
    K = _matrix(weight, "weight").shape[1]
    d = x.device
    return L.LqConv(T, seqs, c, K, _act(activation, ("none", None, "silu")), _dtype_id(x.dtype),
                    _given(weight, _F32, (c, K), "weight", d), _dense(bias, _F32, (c,), "bias", d))


def leapquant_conv_forward(cu_seqlens, x, weight, y, bias=None, activation="silu", X0=None, X=None, stream=None):
    """Short causal convolution of every channel over packed sequences
    (sequence i is tokens cu_seqlens[i] .. cu_seqlens[i+1]-1, int32 on the
    device).  x, y [tokens, channels], strided; weight float32 [channels, width]
    with width 2, 3 or 4, the last one of the token itself; bias float32
    [channels] or None; activation "silu" or "none".  X0 [sequences, width - 1,
    channels] of x's dtype: the inputs before (None: zeros); X the last inputs
    (None: not wanted)."""
    cu, seqs = _offsets(cu_seqlens, _matrix(x, "x").device)
    prm = _conv_params(x, weight, bias, activation, seqs)
    d, dt, s = x.device, x.dtype, (seqs, prm.width - 1, prm.channels)
    _launch(L.load().leapquant_conv_forward, d, stream, prm, cu, _channels(x, dt, x.shape, "x", d),
            _channels(y, dt, x.shape, "y", d), _dense(X0, dt, s, "X0", d), _dense(X, dt, s, "X", d))


def _slots(slots, rows, d):
    return _dense(slots, _I32, (rows,), "slots", d)


def leapquant_conv_step(x, weight, y, X, bias=None, activation="silu", X_out=None, slots=None, stream=None):
    """One token of each row: x, y [rows, channels]; X [n_slots, width - 1,
    channels] the slots' last inputs, updated in place or into X_out (listed
    slots only).  slots int32 [rows] on the device (None: row i is slot i); rows
    whose slot is outside [0, n_slots) are idle; a slot is listed at most once."""
    prm = _conv_params(x, weight, bias, activation, 1)
    d, dt = x.device, x.dtype
    if not isinstance(X, torch.Tensor) or X.dim() != 3:
        raise ValueError("X must be a [n_slots, width - 1, channels] tensor")
    s = (X.shape[0], prm.width - 1, prm.channels)
    to = X if X_out is None else X_out
    _launch(L.load().leapquant_conv_step, d, stream, prm, _slots(slots, x.shape[0], d), X.shape[0],
            _channels(x, dt, x.shape, "x", d), _channels(y, dt, x.shape, "y", d), _dense(X, dt, s, "X", d),
            _dense(to, dt, s, "X_out", d))


def leapquant_conv_workspace(tokens, seqs, channels, width, device="cuda"):
    """Workspace of leapquant_conv_backward with a weight or bias gradient."""
    prm = L.LqConv(int(tokens), int(seqs), int(channels), int(width), L.LQ_ACT_NONE, L.LQ_F32, None, None)
    return torch.empty(_bytes(L.load().leapquant_conv_workspace(ctypes.byref(prm))), dtype=torch.uint8, device=device)


def leapquant_conv_backward(cu_seqlens, x, weight, dy, dx, bias=None, activation="silu", X0=None, dweight=None,
                            dbias=None, dX=None, dX0=None, workspace=None, stream=None):
    """The gradient of leapquant_conv_forward with the same inputs: from dy and
    dX (that of X; None: zeros), writes dx and, where given, dX0, dweight
    (float32 [channels, width]) and dbias (float32 [channels]), which need a
    workspace from leapquant_conv_workspace."""
    cu, seqs = _offsets(cu_seqlens, _matrix(x, "x").device)
    prm = _conv_params(x, weight, bias, activation, seqs)
    d, dt, s = x.device, x.dtype, (seqs, prm.width - 1, prm.channels)
    _launch(L.load().leapquant_conv_backward, d, stream, prm, cu, _channels(x, dt, x.shape, "x", d),
            _channels(dy, dt, x.shape, "dy", d), _channels(dx, dt, x.shape, "dx", d), _dense(X0, dt, s, "X0", d),
            _dense(dX, dt, s, "dX", d), _dense(dX0, dt, s, "dX0", d),
            _dense(dweight, _F32, (prm.channels, prm.width), "dweight", d),
            _dense(dbias, _F32, (prm.channels,), "dbias", d), *_space(workspace, d))


class LeapQuantScan:
    """Parameters and workspace of the selective scan over whole sequences.

    Serves calls of at most max_tokens tokens in at most max_seqs sequences with
    `channels` channels of `states` (8, 16 or 32) states, `groups` of which share
    B and C, in `dtype`.  softplus: steps are log(1 + e^(dt + dt_bias)) instead of
    dt + dt_bias.  save: for forward calls that a backward call follows; the
    workspace then holds what the backward call reads, so a plan serves one
    forward and its backward calls at a time (a backward call whose tokens or
    sequences are not those of the plan's last forward call is refused).  Calls
    that may run at the same time, and captured graphs that may, need a plan
    each; a plan outlives the work that was launched with it, and every replay of
    a graph that holds its calls.
    """

    def __init__(self, max_tokens, max_seqs, channels, states, groups=1, dtype=torch.bfloat16, device="cuda",
                 softplus=True, save=False):
        self.max_tokens, self.max_seqs = int(max_tokens), int(max_seqs)
        self.channels, self.states, self.groups = int(channels), int(states), int(groups)
        self.dtype, self.softplus, self.save = dtype, bool(softplus), bool(save)
        prm = self.params(self.max_tokens, self.max_seqs)
        size = _bytes(L.load().leapquant_scan_workspace(ctypes.byref(prm), int(self.save)))
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)
        self.device = self.workspace.device   # with its index resolved
        self._saved = None   # tokens and sequences of the forward call that the workspace holds

    def params(self, tokens, seqs, A=None, D=None, dt_bias=None):
        return _scan_params(tokens, seqs, self.channels, self.states, self.groups, self.dtype, self.softplus, A, D,
                            dt_bias)

    def _call(self, cu_seqlens, x, A, D, dt_bias):
        """(parameters, cu_seqlens pointer, tokens, sequences) of a call."""
        T = _matrix(x, "x").shape[0]
        cu, seqs = _offsets(cu_seqlens, self.device)
        if T > self.max_tokens or seqs > self.max_seqs:
            raise ValueError(f"{T} tokens in {seqs} sequences: the plan is for {self.max_tokens} in {self.max_seqs}")
        return self.params(T, seqs, *_scan_weights(self.channels, self.states, A, D, dt_bias, self.device)), cu, T, seqs

    def _space(self):
        return ctypes.c_void_p(self.workspace.data_ptr() or None), self.workspace.numel()


def _scan_params(tokens, seqs, channels, states, groups, dtype, softplus, A, D, dt_bias):
    return L.LqScan(int(tokens), int(seqs), channels, states, groups, _dtype_id(dtype),
                    L.LQ_SCAN_SOFTPLUS if softplus else 0, A, D, dt_bias)


def _scan_weights(channels, states, A, D, dt_bias, d):
    return (_given(A, _F32, (channels, states), "A", d), _dense(D, _F32, (channels,), "D", d),
            _dense(dt_bias, _F32, (channels,), "dt_bias", d))


def _scan_inputs(T, channels, states, groups, dt, d, x, dt_in, B, C, z):
    wide, low = (T, channels), (T, groups, states)
    return [_channels(x, dt, wide, "x", d), _channels(dt_in, dt, wide, "dt", d), _rows(B, dt, low, "B", d),
            _rows(C, dt, low, "C", d), _channels(z, dt, wide, "z", d)]


def leapquant_scan_forward(plan, cu_seqlens, x, dt, A, B, C, y, D=None, dt_bias=None, z=None, S0=None, S=None,
                           stream=None):
    """The selective scan over packed sequences (sequence i is tokens
    cu_seqlens[i] .. cu_seqlens[i+1]-1, int32 on the device): h = exp(d A) h + d B x,
    y = (sum of C h + D x) silu(z), with d from dt and dt_bias.  x, dt, z (None: no
    gate), y [tokens, channels] and B, C [tokens, groups, states] of plan.dtype,
    strided; A [channels, states], D and dt_bias [channels] (None: zeros) float32.
    States float32 [sequences, channels, states]: S0 before (None: zeros), S after
    (None: not wanted; may be S0)."""
    prm, cu, T, seqs = plan._call(cu_seqlens, x, A, D, dt_bias)
    d, c, n, dtype = plan.device, plan.channels, plan.states, plan.dtype
    _launch(L.load().leapquant_scan_forward, d, stream, prm, cu,
            *_scan_inputs(T, c, n, plan.groups, dtype, d, x, dt, B, C, z), _channels(y, dtype, (T, c), "y", d),
            _dense(S0, _F32, (seqs, c, n), "S0", d), _dense(S, _F32, (seqs, c, n), "S", d), *plan._space(),
            int(plan.save))
    if plan.save:
        plan._saved = T, seqs


def leapquant_scan_step(x, dt, A, B, C, y, S, D=None, dt_bias=None, z=None, S_out=None, slots=None, softplus=True,
                        stream=None):
    """One token of each row: x, dt, z, y [rows, channels], B, C [rows, groups,
    states]; S float32 [n_slots, channels, states] the slots' states, updated in
    place or into S_out (listed slots only).  slots int32 [rows] on the device
    (None: row i is slot i); rows whose slot is outside [0, n_slots) are idle; a
    slot is listed at most once.  The rest as in leapquant_scan_forward."""
    T, c = _matrix(x, "x").shape
    if not isinstance(S, torch.Tensor) or S.dim() != 3:
        raise ValueError("S must be a [n_slots, channels, states] tensor")
    if not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("B must be a [rows, groups, states] tensor")
    d, g, n = x.device, B.shape[1], B.shape[2]
    prm = _scan_params(T, 1, c, n, g, x.dtype, softplus, *_scan_weights(c, n, A, D, dt_bias, d))
    s = (S.shape[0], c, n)
    to = S if S_out is None else S_out
    _launch(L.load().leapquant_scan_step, d, stream, prm, _slots(slots, T, d), S.shape[0],
            *_scan_inputs(T, c, n, g, x.dtype, d, x, dt, B, C, z), _channels(y, x.dtype, (T, c), "y", d),
            _given(S, _F32, s, "S", d), _given(to, _F32, s, "S_out", d))


def leapquant_scan_backward(plan, cu_seqlens, x, dt, A, B, C, dy, dx, ddt, dA, dB, dC, D=None, dt_bias=None, z=None,
                            dD=None, ddt_bias=None, dz=None, dS=None, dS0=None, stream=None):
    """The gradient of the plan's last leapquant_scan_forward (same cu_seqlens and
    inputs; a plan with save): from dy and dS, the gradients of y and S (None:
    zeros), writes dx, ddt, dA, dB, dC and, where given, dD, ddt_bias and dS0 (may
    be dS), shaped as their inputs; dz with a gate."""
    if not plan.save:
        raise ValueError("the plan was made without save")
    if plan._saved is None:
        raise ValueError("the plan holds no forward call")
    prm, cu, T, seqs = plan._call(cu_seqlens, x, A, D, dt_bias)
    if plan._saved != (T, seqs):
        raise ValueError("the plan holds a forward call of %d tokens in %d sequences, " % plan._saved +
                         f"not of {T} in {seqs}")
    if (z is None) != (dz is None):
        raise ValueError("z and dz come together")
    if (dD is not None and D is None) or (ddt_bias is not None and dt_bias is None):
        raise ValueError("dD comes with D, ddt_bias with dt_bias")
    d, c, n, g, dtype = plan.device, plan.channels, plan.states, plan.groups, plan.dtype
    wide, low = (T, c), (T, g, n)
    _launch(L.load().leapquant_scan_backward, d, stream, prm, cu,
            *_scan_inputs(T, c, n, g, dtype, d, x, dt, B, C, z), _channels(dy, dtype, wide, "dy", d),
            _channels(dx, dtype, wide, "dx", d), _channels(ddt, dtype, wide, "ddt", d), _rows(dB, dtype, low, "dB", d),
            _rows(dC, dtype, low, "dC", d), _channels(dz, dtype, wide, "dz", d), _given(dA, _F32, (c, n), "dA", d),
            _dense(dD, _F32, (c,), "dD", d), _dense(ddt_bias, _F32, (c,), "ddt_bias", d),
            _dense(dS, _F32, (seqs, c, n), "dS", d), _dense(dS0, _F32, (seqs, c, n), "dS0", d), *plan._space())


def _norm_params(a, stream_dtype, gate, z, scale, out_norm, out_weight, in_weight, eps):
    if not isinstance(a, torch.Tensor) or a.dim() != 3:
        raise ValueError("a must be a [tokens, heads, dim] tensor")
    gate = _act(gate, _ACTS) if z is not None else L.LQ_ACT_NONE
    if z is not None and gate == L.LQ_ACT_NONE:
        raise ValueError("z needs a gate, \"silu\" or \"sigmoid\"")
    if out_weight is not None and not out_norm:
        raise ValueError("out_weight needs out_norm")
    T, heads, dim = a.shape
    return L.LqBlockNorm(T, heads, dim, _dtype_id(a.dtype), _dtype_id(stream_dtype), gate, int(bool(out_norm)),
                         float(eps), float(scale), _dense(out_weight, _F32, (dim,), "out_weight", a.device),
                         _dense(in_weight, _F32, (dim,), "in_weight", a.device))


def _stream_dtype(a, *arrays):
    """The residual stream's dtype: that of the first of its arrays that is given, otherwise a's."""
    return next((x.dtype for x in arrays if isinstance(x, torch.Tensor)), a.dtype)


def leapquant_block_norm(a, h=None, y=None, z=None, res=None, gate="silu", scale=1.0, out_norm=False, out_weight=None,
                         in_weight=None, eps=1e-6, stream=None):
    """Norms before and after a block, with its gate and residual scale, of rows
    of dim values: n = out_weight * a / rms(a) with out_norm (otherwise a), u = n *
    gate(z) with z ("silu" or "sigmoid"), h = res + scale * u (without res: scale *
    u), y = in_weight * h / rms(h).  a, z, y [tokens, heads, dim] of one dtype, res
    and h of the same or float32, strided; weights float32 [dim] (None: ones).  h
    and y are written where given, at least one; they may be a or res itself."""
    if not isinstance(a, torch.Tensor):
        raise TypeError("a must be a torch.Tensor")
    wide = _stream_dtype(a, res, h)
    prm = _norm_params(a, wide, gate, z, scale, out_norm, out_weight, in_weight, eps)
    if h is None and y is None:
        raise ValueError("h or y must be given")
    d, dt, s = a.device, a.dtype, a.shape
    _launch(L.load().leapquant_block_norm, d, stream, prm, _heads(a, dt, s, "a", d), _heads(z, dt, s, "z", d),
            _heads(res, wide, s, "res", d), _heads(h, wide, s, "h", d), _heads(y, dt, s, "y", d))


def leapquant_block_norm_workspace(tokens, heads, dim, device="cuda"):
    """Workspace of leapquant_block_norm_backward with a weight gradient."""
    n = _bytes(L.load().leapquant_block_norm_workspace(int(tokens), int(heads), int(dim)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def leapquant_block_norm_backward(a, da, dh=None, dy=None, z=None, res=None, gate="silu", scale=1.0, out_norm=False,
                                  out_weight=None, in_weight=None, eps=1e-6, dz=None, dres=None, dout_weight=None,
                                  din_weight=None, workspace=None, stream=None):
    """The gradient of leapquant_block_norm with the same inputs: from dh and dy
    (at least one; None: zeros), writes da, dz with a gate and, where given, dres
    (may be dh), dout_weight and din_weight (float32 [dim], which need a workspace
    from leapquant_block_norm_workspace)."""
    if not isinstance(a, torch.Tensor):
        raise TypeError("a must be a torch.Tensor")
    wide = _stream_dtype(a, res, dh, dres)
    prm = _norm_params(a, wide, gate, z, scale, out_norm, out_weight, in_weight, eps)
    if dh is None and dy is None:
        raise ValueError("dh or dy must be given")
    if (z is None) != (dz is None):
        raise ValueError("z and dz come together")
    if (dres is not None and res is None) or (dout_weight is not None and not out_norm) or (
            din_weight is not None and dy is None):
        raise ValueError("dres comes with res, dout_weight with out_norm, din_weight with dy")
    d, dt, s = a.device, a.dtype, a.shape
    w = (s[2],)
    _launch(L.load().leapquant_block_norm_backward, d, stream, prm, _heads(a, dt, s, "a", d), _heads(z, dt, s, "z", d),
            _heads(res, wide, s, "res", d), _heads(dh, wide, s, "dh", d), _heads(dy, dt, s, "dy", d),
            _heads(da, dt, s, "da", d), _heads(dz, dt, s, "dz", d), _heads(dres, wide, s, "dres", d),
            _dense(dout_weight, _F32, w, "dout_weight", d), _dense(din_weight, _F32, w, "din_weight", d),
            *_space(workspace, d))
