"""Python binding of the sequence operators of the C ABI (argument marshalling
only): the recurrence over whole sequences with its gradient, and the norm of
query and key heads.  See include/leapquant.h for the semantics of each call.
"""
import ctypes

import torch

from . import _lib as L
from .api import _F32, _I32, _gate_id, _ptr, _stream

_DTYPES = {torch.float32: L.LQ_F32, torch.bfloat16: L.LQ_BF16, torch.float16: L.LQ_F16}
_NORMS = {"l2": L.LQ_NORM_L2, "rms": L.LQ_NORM_RMS, L.LQ_NORM_L2: L.LQ_NORM_L2, L.LQ_NORM_RMS: L.LQ_NORM_RMS}
# The current stream's handle without a Stream object: a call of 10 us, 12.5 with
# one.  No public name of torch's, so a version that lacks it takes the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dtype_id(dtype):
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    return _DTYPES[dtype]


def _rows(x, dtype, shape, name, device):
    """A strided [tokens, heads(, 128)] tensor as lq_rows."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device != device:
        raise ValueError(f"{name} must be in device memory" if x.device.type != "cuda" else
                         f"{name} is on {x.device}, the call on {device}")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    strides = x.stride()
    if len(strides) == 3 and strides[2] != 1 and x.numel():
        raise ValueError(f"{name}: the values of a head must be contiguous")
    return L.LqRows(x.data_ptr() or None, strides[0], strides[1])


def _launch(fn, device, stream, *args):
    """The call on its device, with the stream's handle as the last argument."""
    if device.type != "cuda":
        raise ValueError("the call's tensors must be in device memory")
    if torch.cuda.current_device() == device.index:
        raw = stream is None and _raw_stream is not None
        handle = _raw_stream(device.index) if raw else _stream(stream, device)
        return L.check(fn(*args, handle))
    with torch.cuda.device(device):
        L.check(fn(*args, _stream(stream, device)))


def _states(x, n, name, device):
    return None if x is None else _ptr(x, _F32, (n, 128, 128), name, device)


def _bytes(n):
    """A workspace size, or the error it stands for."""
    if n < 0:
        L.check(int(n))
    return n


class LeapQuantSequence:
    """Parameters and workspace of the calls over whole sequences.

    Serves calls of at most max_tokens tokens in at most max_seqs sequences,
    with heads_k query and key heads and heads_v value heads of `dtype`.
    save: for forward calls that a backward call follows; the workspace then
    holds what the backward call reads, so a plan serves one forward and its
    backward calls at a time (a backward call whose tokens or sequences are not
    those of the plan's last forward call, also into a capture, is refused).
    Calls that may run at the same time, and
    captured graphs that may, need a plan each; a plan outlives the work that
    was launched with it, and every replay of a graph that holds its calls.
    """

    def __init__(self, max_tokens, max_seqs, heads_k, heads_v, gate="gdn", dtype=torch.bfloat16, device="cuda",
                 flags=0, save=False):
        self.max_tokens, self.max_seqs = int(max_tokens), int(max_seqs)
        self.heads_k, self.heads_v = int(heads_k), int(heads_v)
        self.gate, self.dtype, self.flags, self.save = _gate_id(gate), dtype, int(flags), bool(save)
        prm = self.params(self.max_tokens, self.max_seqs)
        size = _bytes(L.load().leapquant_sequence_workspace(ctypes.byref(prm), int(self.save)))
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)
        self.device = self.workspace.device   # with its index resolved
        self._saved = None   # tokens and sequences of the forward call that the workspace holds

    def params(self, tokens, seqs):
        return L.LqSequence(int(tokens), int(seqs), self.heads_k, self.heads_v, 128, 128, self.gate, self.flags,
                            _dtype_id(self.dtype))

    def _call(self, cu_seqlens, q):
        """(parameters, cu_seqlens pointer, tokens, sequences) of a call."""
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a [tokens, heads_k, 128] tensor")
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor of sequences + 1 offsets")
        tokens, seqs = q.shape[0], cu_seqlens.numel() - 1
        if tokens > self.max_tokens or seqs > self.max_seqs:
            raise ValueError(f"{tokens} tokens in {seqs} sequences: the plan is for {self.max_tokens} in "
                             f"{self.max_seqs}")
        return (self.params(tokens, seqs), _ptr(cu_seqlens, _I32, (seqs + 1,), "cu_seqlens", self.device),
                tokens, seqs)

    def _space(self):
        return ctypes.c_void_p(self.workspace.data_ptr() or None), self.workspace.numel()


def leapquant_sequence_forward(plan, cu_seqlens, q, k, v, beta, alpha, o, S0=None, S=None, stream=None):
    """The recurrence over packed sequences: sequence i is tokens
    cu_seqlens[i] .. cu_seqlens[i+1]-1 (int32 on the device).  q, k [tokens,
    heads_k, 128], v, o [tokens, heads_v, 128] of plan.dtype (strided, the
    last axis contiguous); beta [tokens, heads_v]; alpha [tokens, heads_v]
    (gdn) or [tokens, heads_v, 128] (kda), float32.  States float32
    [sequences * heads_v, 128, 128]: S0 before (None: zeros), S after (None:
    not wanted; may be S0).  One long sequence among many short ones is better
    a call of its own (include/leapquant.h says which form a call takes)."""
    prm, cu, T, seqs = plan._call(cu_seqlens, q)
    d, hk, hv, dt = plan.device, plan.heads_k, plan.heads_v, plan.dtype
    ashape = (T, hv) if plan.gate == L.LQ_GATE_GDN else (T, hv, 128)
    args = [_rows(q, dt, (T, hk, 128), "q", d), _rows(k, dt, (T, hk, 128), "k", d),
            _rows(v, dt, (T, hv, 128), "v", d), _rows(beta, _F32, (T, hv), "beta", d),
            _rows(alpha, _F32, ashape, "alpha", d), _rows(o, dt, (T, hv, 128), "o", d),
            _states(S0, seqs * hv, "S0", d), _states(S, seqs * hv, "S", d)]
    _launch(L.load().leapquant_sequence_forward, d, stream, prm, cu, *args, *plan._space(), int(plan.save))
    if plan.save:
        plan._saved = T, seqs


def leapquant_sequence_backward(plan, cu_seqlens, q, k, beta, alpha, do, dq, dk, dv, dbeta, dalpha, dS=None,
                                dS0=None, stream=None):
    """The gradient of the plan's last leapquant_sequence_forward (same
    cu_seqlens, q, k, beta and alpha; a plan with save): from do, the
    gradient of o, and dS, that of S (None: zeros), writes dq, dk, dv, dbeta,
    dalpha and dS0 (None: not wanted; may be dS), shaped as their inputs."""
    if not plan.save:
        raise ValueError("the plan was made without save")
    if plan._saved is None:
        raise ValueError("the plan holds no forward call")
    prm, cu, T, seqs = plan._call(cu_seqlens, q)
    if plan._saved != (T, seqs):
        raise ValueError("the plan holds a forward call of %d tokens in %d sequences, " % plan._saved +
                         f"not of {T} in {seqs}")
    d, hk, hv, dt = plan.device, plan.heads_k, plan.heads_v, plan.dtype
    args = [_rows(q, dt, (T, hk, 128), "q", d), _rows(k, dt, (T, hk, 128), "k", d),
            _rows(beta, _F32, (T, hv), "beta", d), _rows(alpha, _F32, (T, hv), "alpha", d),
            _rows(do, dt, (T, hv, 128), "do", d), _states(dS, seqs * hv, "dS", d),
            _rows(dq, dt, (T, hk, 128), "dq", d), _rows(dk, dt, (T, hk, 128), "dk", d),
            _rows(dv, dt, (T, hv, 128), "dv", d), _rows(dbeta, _F32, (T, hv), "dbeta", d),
            _rows(dalpha, _F32, (T, hv), "dalpha", d), _states(dS0, seqs * hv, "dS0", d)]
    _launch(L.load().leapquant_sequence_backward, d, stream, prm, cu, *args, *plan._space())


def _norm_params(q, k, out, norm, eps, q_weight, k_weight, q_scale, positions, inv_freq, interleaved):
    if norm not in _NORMS:
        raise ValueError(f"unknown norm {norm!r}")
    for x, name in ((q, "q"), (k, "k")):
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            raise ValueError(f"{name} must be a [tokens, heads, 128] tensor")
    d, T = q.device, q.shape[0]
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    rot, pos, freq = 0, None, None
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a 1-D float64 tensor of rot / 2 frequencies")
        rot = 2 * inv_freq.numel()
        pos = _ptr(positions, torch.int64, (T,), "positions", d)
        freq = _ptr(inv_freq, torch.float64, (rot // 2,), "inv_freq", d)
    wq, wk = (None if w is None else _ptr(w, _F32, (128,), n, d)
              for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")))
    return L.LqHeadNorm(T, q.shape[1], k.shape[1], 128, _NORMS[norm], _dtype_id(q.dtype), _dtype_id(out.dtype), rot,
                        int(bool(interleaved)), float(eps), float(q_scale), wq, wk, pos, freq)


def leapquant_head_norm(q, k, q_out, k_out, norm="l2", eps=1e-6, q_weight=None, k_weight=None, q_scale=1.0,
                        positions=None, inv_freq=None, interleaved=False, stream=None):
    """Norm of every query and key head ("l2": unit norm; "rms"), times the
    weights (float32 [128]) and, for queries, q_scale, with the first
    2 * len(inv_freq) values rotated by positions (int64 [tokens]) times
    inv_freq (float64).  q, q_out [tokens, heads_q, 128], k, k_out [tokens,
    heads_k, 128], strided; q and k of one dtype, the outputs of one (it may
    differ: float32 for the decode calls)."""
    prm = _norm_params(q, k, q_out, norm, eps, q_weight, k_weight, q_scale, positions, inv_freq, interleaved)
    d, T, shape_q, shape_k = q.device, q.shape[0], (q.shape[0], q.shape[1], 128), (q.shape[0], k.shape[1], 128)
    args = [_rows(q, q.dtype, shape_q, "q", d), _rows(k, q.dtype, shape_k, "k", d),
            _rows(q_out, q_out.dtype, shape_q, "q_out", d), _rows(k_out, q_out.dtype, shape_k, "k_out", d)]
    _launch(L.load().leapquant_head_norm, d, stream, prm, *args)


def leapquant_head_norm_workspace(tokens, heads_q, heads_k, device="cuda"):
    """Workspace of leapquant_head_norm_backward with weight gradients."""
    n = _bytes(L.load().leapquant_head_norm_workspace(int(tokens), int(heads_q), int(heads_k)))
    return torch.empty(n, dtype=torch.uint8, device=device)


def leapquant_head_norm_backward(q, k, dq_out, dk_out, dq, dk, norm="l2", eps=1e-6, q_weight=None, k_weight=None,
                                 q_scale=1.0, positions=None, inv_freq=None, interleaved=False, dq_weight=None,
                                 dk_weight=None, workspace=None, stream=None):
    """The gradient of leapquant_head_norm with the same q, k and parameters:
    from dq_out and dk_out, writes dq and dk (dtype of q and k) and, where
    given, dq_weight and dk_weight (float32 [128], which need a workspace
    from leapquant_head_norm_workspace)."""
    prm = _norm_params(q, k, dq_out, norm, eps, q_weight, k_weight, q_scale, positions, inv_freq, interleaved)
    d, shape_q, shape_k = q.device, (q.shape[0], q.shape[1], 128), (q.shape[0], k.shape[1], 128)
    args = [_rows(q, q.dtype, shape_q, "q", d), _rows(k, q.dtype, shape_k, "k", d),
            _rows(dq_out, dq_out.dtype, shape_q, "dq_out", d), _rows(dk_out, dq_out.dtype, shape_k, "dk_out", d),
            _rows(dq, q.dtype, shape_q, "dq", d), _rows(dk, q.dtype, shape_k, "dk", d)]
    args += [None if w is None else _ptr(w, _F32, (128,), n, d)
             for w, n in ((dq_weight, "dq_weight"), (dk_weight, "dk_weight"))]
    if workspace is None:
        args += [None, 0]
    else:
        args += [_ptr(workspace, torch.uint8, (workspace.numel(),), "workspace", d), workspace.numel()]
    _launch(L.load().leapquant_head_norm_backward, d, stream, prm, *args)
