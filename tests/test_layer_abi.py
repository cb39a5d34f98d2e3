"""Refusals of the convolution, scan and block norm entry points (CPU): every
call here is rejected by host-side validation before any launch, so fake
addresses are safe; the same checks under AddressSanitizer and UBSan, and from
plain C, are in the last tests."""
import ctypes
import os
import subprocess

import pytest
import torch

import recurrent_state_quant_amd as lq
from recurrent_state_quant_amd import _lib as L
from recurrent_state_quant_amd import build as B

BASE = 0x7F0000000000  # never dereferenced
MB = 1 << 20
T, SEQS, CH, N, G = 100, 3, 64, 16, 2


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _addr(i):
    return BASE + i * 64 * MB


def _rows(i, width, off=0, ts=None):
    return L.LqRows(_addr(i) + off, width if ts is None else ts, 0)


def _heads(i, heads, width, off=0):
    return L.LqRows(_addr(i) + off, heads * width, width)


def _by(x):
    return None if x is None else ctypes.byref(x)


# ---------------------------------------------------------------- convolution
def _cv(**kw):
    d = dict(tokens=T, seqs=SEQS, channels=CH, width=4, activation=L.LQ_ACT_SILU, dtype=L.LQ_BF16, weight=_addr(20),
             bias=_addr(21))
    d.update(kw)
    return L.LqConv(*[d[f] for f, _ in L.LqConv._fields_])


def _conv(lib, cv=None, **kw):
    a = dict(cu=_addr(0), x=_rows(1, CH), y=_rows(2, CH), X0=_addr(3), X=_addr(4))
    a.update(kw)
    return lib.leapquant_conv_forward(_by(cv or _cv()), a["cu"], _by(a["x"]), _by(a["y"]), a["X0"], a["X"], None)


def _conv_step(lib, cv=None, **kw):
    a = dict(slots=_addr(0), n=200, x=_rows(1, CH), y=_rows(2, CH), X0=_addr(3), X=_addr(4))
    a.update(kw)
    return lib.leapquant_conv_step(_by(cv or _cv()), a["slots"], a["n"], _by(a["x"]), _by(a["y"]), a["X0"], a["X"], None)


def _conv_back(lib, cv=None, **kw):
    a = dict(cu=_addr(0), x=_rows(1, CH), dy=_rows(2, CH), dx=_rows(5, CH), X0=_addr(3), dX=_addr(4), dX0=_addr(6),
             dw=_addr(7), db=_addr(8), ws=_addr(9), nbytes=1 << 30)
    a.update(kw)
    return lib.leapquant_conv_backward(_by(cv or _cv()), a["cu"], _by(a["x"]), _by(a["dy"]), _by(a["dx"]), a["X0"],
                                       a["dX"], a["dX0"], a["dw"], a["db"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(channels=0), dict(channels=(1 << 20) + 1),
                                dict(activation=2), dict(activation=-1), dict(dtype=3),
                                dict(tokens=1 << 30, channels=1 << 20)])
def test_conv_shapes(lib, kw):
    for call in (_conv, _conv_step, _conv_back):
        assert call(lib, _cv(**kw)) == L.LQ_ERR_SHAPE
    assert lib.leapquant_conv_workspace(_by(_cv(**kw))) == L.LQ_ERR_SHAPE


def test_conv_other_refusals(lib):
    for w in (1, 5, 0):
        for call in (_conv, _conv_step, _conv_back):
            assert call(lib, _cv(width=w)) == L.LQ_ERR_UNSUPPORTED
    for seqs in (0, -1, 1 << 30):
        assert _conv(lib, _cv(seqs=seqs)) == L.LQ_ERR_SHAPE
        assert _conv_back(lib, _cv(seqs=seqs)) == L.LQ_ERR_SHAPE
    for name in ("cu", "x", "y"):
        assert _conv(lib, **{name: None}) == L.LQ_ERR_NULL
    assert _conv(lib, x=L.LqRows(None, CH, 0)) == L.LQ_ERR_NULL
    assert _conv(lib, _cv(weight=None)) == L.LQ_ERR_NULL
    assert _conv(lib, cu=_addr(0) + 2) == L.LQ_ERR_ALIGN
    assert _conv(lib, x=_rows(1, CH, 1)) == L.LQ_ERR_ALIGN
    assert _conv(lib, _cv(dtype=L.LQ_F32), x=_rows(1, CH, 2)) == L.LQ_ERR_ALIGN
    assert _conv(lib, X=_addr(4) + 1) == L.LQ_ERR_ALIGN
    assert _conv(lib, _cv(bias=_addr(21) + 2)) == L.LQ_ERR_ALIGN
    assert _conv(lib, x=_rows(1, CH, ts=-CH)) == L.LQ_ERR_SHAPE
    assert _conv(lib, y=_rows(2, CH, ts=CH - 1)) == L.LQ_ERR_SHAPE   # an output's rows overlap
    assert _conv(lib, y=_rows(2, CH, ts=0)) == L.LQ_ERR_SHAPE
    for kw in (dict(y=_rows(1, CH)), dict(X=_addr(3)), dict(X=_addr(3) + 128), dict(X=_addr(1)), dict(y=_rows(0, CH)),
               dict(y=_rows(20, CH)), dict(X=_addr(2) + 64), dict(y=_rows(1, CH, 64, ts=CH + 32), x=_rows(1, CH, ts=CH + 32))):
        assert _conv(lib, **kw) == L.LQ_ERR_ALIAS, kw


def test_conv_step_refusals(lib):
    for name in ("x", "y", "X0", "X"):
        assert _conv_step(lib, **{name: None}) == L.LQ_ERR_NULL
    assert _conv_step(lib, n=0) == L.LQ_ERR_SHAPE
    assert _conv_step(lib, slots=None, n=T - 1) == L.LQ_ERR_SHAPE
    assert _conv_step(lib, slots=_addr(0) + 1) == L.LQ_ERR_ALIGN
    assert _conv_step(lib, X=_addr(3) + 2) == L.LQ_ERR_ALIAS
    assert _conv_step(lib, y=_rows(3, CH)) == L.LQ_ERR_ALIAS
    assert _conv_step(lib, X0=_addr(0), X=_addr(0)) == L.LQ_ERR_ALIAS


def test_conv_backward_refusals(lib):
    for name in ("cu", "x", "dy", "dx", "ws"):
        assert _conv_back(lib, **{name: None}) == L.LQ_ERR_NULL
    assert _conv_back(lib, nbytes=100) == L.LQ_ERR_SHAPE
    assert _conv_back(lib, ws=_addr(9) + 8) == L.LQ_ERR_ALIGN
    assert _conv_back(lib, dw=_addr(7) + 2) == L.LQ_ERR_ALIGN
    for kw in (dict(dx=_rows(2, CH)), dict(dX0=_addr(4)), dict(dX0=_addr(3)), dict(dw=_addr(20)), dict(db=_addr(7) + 16),
               dict(ws=_addr(5)), dict(dw=_addr(9) + 64)):
        assert _conv_back(lib, **kw) == L.LQ_ERR_ALIAS, kw


def test_conv_workspace_covers_smaller_calls(lib):
    size = lambda t: lib.leapquant_conv_workspace(_by(_cv(tokens=t)))  # noqa: E731
    for most in (1, 127, 4000, 32768, 40000, 300000, 1 << 23):
        for t in {1, most // 3, most // 2, most - 1, most} - {0}:
            # a null output is refused after the workspace's size is (dx shares memory with dy)
            assert _conv_back(lib, _cv(tokens=t), nbytes=size(most), dx=_rows(2, CH)) == L.LQ_ERR_ALIAS
    assert size(0) == 0


# ---------------------------------------------------------------- scan
def _sc(**kw):
    d = dict(tokens=T, seqs=SEQS, channels=CH, states=N, groups=G, dtype=L.LQ_BF16, flags=L.LQ_SCAN_SOFTPLUS, A=_addr(20),
             D=_addr(21), dt_bias=_addr(22))
    d.update(kw)
    return L.LqScan(*[d[f] for f, _ in L.LqScan._fields_])


SCAN_IN = dict(x=_rows(1, CH), dt=_rows(2, CH), B=_heads(3, G, N), C=_heads(4, G, N), z=_rows(5, CH))


def _scan(lib, sc=None, save=0, **kw):
    a = dict(SCAN_IN, cu=_addr(0), y=_rows(6, CH), S0=_addr(7), S=_addr(8), ws=_addr(9), nbytes=1 << 40)
    a.update(kw)
    r = [_by(a[m]) for m in ("x", "dt", "B", "C", "z", "y")]
    return lib.leapquant_scan_forward(_by(sc or _sc()), a["cu"], *r, a["S0"], a["S"], a["ws"], a["nbytes"], save, None)


def _scan_step(lib, sc=None, **kw):
    a = dict(SCAN_IN, slots=_addr(0), n=200, y=_rows(6, CH), S0=_addr(7), S=_addr(8))
    a.update(kw)
    r = [_by(a[m]) for m in ("x", "dt", "B", "C", "z", "y")]
    return lib.leapquant_scan_step(_by(sc or _sc()), a["slots"], a["n"], *r, a["S0"], a["S"], None)


def _scan_back(lib, sc=None, **kw):
    a = dict(SCAN_IN, cu=_addr(0), dy=_rows(6, CH), dx=_rows(10, CH), ddt=_rows(11, CH), dB=_heads(12, G, N),
             dC=_heads(13, G, N), dz=_rows(14, CH), dA=_addr(15), dD=_addr(16), db=_addr(17), dS=_addr(7), dS0=_addr(8),
             ws=_addr(9), nbytes=1 << 40)
    a.update(kw)
    r = [_by(a[m]) for m in ("x", "dt", "B", "C", "z", "dy", "dx", "ddt", "dB", "dC", "dz")]
    return lib.leapquant_scan_backward(_by(sc or _sc()), a["cu"], *r, a["dA"], a["dD"], a["db"], a["dS"], a["dS0"],
                                       a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(channels=0), dict(channels=1 << 21),
                                dict(groups=0), dict(groups=3), dict(groups=1 << 17, channels=1 << 17), dict(flags=2),
                                dict(dtype=3), dict(tokens=1 << 30, channels=1 << 20)])
def test_scan_shapes(lib, kw):
    for call in (_scan, _scan_step, _scan_back):
        assert call(lib, _sc(**kw)) == L.LQ_ERR_SHAPE
    assert lib.leapquant_scan_workspace(_by(_sc(**kw)), 0) == L.LQ_ERR_SHAPE


@pytest.mark.parametrize("states", [0, 4, 12, 64])
def test_scan_states(lib, states):
    for call in (_scan, _scan_step, _scan_back):
        assert call(lib, _sc(states=states)) == L.LQ_ERR_UNSUPPORTED


def test_scan_other_refusals(lib):
    for seqs in (0, -5, 1 << 30):
        assert _scan(lib, _sc(seqs=seqs)) == L.LQ_ERR_SHAPE
        assert _scan_back(lib, _sc(seqs=seqs)) == L.LQ_ERR_SHAPE
    for name in ("cu", "x", "dt", "B", "C", "y", "ws"):
        assert _scan(lib, **{name: None}) == L.LQ_ERR_NULL
        if name not in ("cu", "ws"):
            assert _scan(lib, **{name: L.LqRows(None, CH, N)}) == L.LQ_ERR_NULL
    assert _scan(lib, _sc(A=None)) == L.LQ_ERR_NULL
    assert _scan(lib, z=L.LqRows(None, CH, 0)) == L.LQ_ERR_NULL
    for kw in (dict(x=_rows(1, CH, 1)), dict(B=_heads(3, G, N, 8)), dict(C=L.LqRows(_addr(4), 36, 16)), dict(cu=_addr(0) + 2),
               dict(B=L.LqRows(_addr(3), 64, 20)), dict(S0=_addr(7) + 8), dict(S=_addr(8) + 4), dict(ws=_addr(9) + 8)):
        assert _scan(lib, **kw) == L.LQ_ERR_ALIGN, kw
    assert _scan(lib, _sc(A=_addr(20) + 4)) == L.LQ_ERR_ALIGN
    assert _scan(lib, _sc(D=_addr(21) + 2)) == L.LQ_ERR_ALIGN
    for kw in (dict(y=_rows(6, CH, ts=CH - 2)), dict(x=_rows(1, CH, ts=-1)), dict(nbytes=64), dict(dt=_rows(2, CH, ts=1 << 50))):
        assert _scan(lib, **kw) == L.LQ_ERR_SHAPE, kw
    for kw in (dict(y=_rows(1, CH)), dict(y=_rows(3, CH)), dict(S=_addr(7) + 64), dict(S=_addr(6)), dict(ws=_addr(5)),
               dict(S=_addr(20)), dict(y=_rows(22, CH)), dict(ws=_addr(0)), dict(ws=_addr(8))):
        assert _scan(lib, **kw) == L.LQ_ERR_ALIAS, kw


def test_scan_step_refusals(lib):
    for name in ("x", "dt", "B", "C", "y", "S0", "S"):
        assert _scan_step(lib, **{name: None}) == L.LQ_ERR_NULL
    assert _scan_step(lib, n=0) == L.LQ_ERR_SHAPE
    assert _scan_step(lib, slots=None, n=T - 1) == L.LQ_ERR_SHAPE
    assert _scan_step(lib, slots=_addr(0) + 2) == L.LQ_ERR_ALIGN
    assert _scan_step(lib, S=_addr(8) + 8) == L.LQ_ERR_ALIGN
    assert _scan_step(lib, S=_addr(7) + 64) == L.LQ_ERR_ALIAS
    assert _scan_step(lib, y=_rows(5, CH)) == L.LQ_ERR_ALIAS
    assert _scan_step(lib, S0=_addr(0), S=_addr(0)) == L.LQ_ERR_ALIAS


def test_scan_backward_refusals(lib):
    for name in ("cu", "x", "dt", "B", "C", "dy", "dx", "ddt", "dB", "dC", "dz", "dA", "ws"):
        assert _scan_back(lib, **{name: None}) == L.LQ_ERR_NULL
    assert _scan_back(lib, z=None) == L.LQ_ERR_NULL             # dz without z
    assert _scan_back(lib, _sc(D=None)) == L.LQ_ERR_NULL        # dD without D
    assert _scan_back(lib, _sc(dt_bias=None)) == L.LQ_ERR_NULL
    assert _scan_back(lib, nbytes=1000) == L.LQ_ERR_SHAPE
    for kw in (dict(dA=_addr(15) + 4), dict(dD=_addr(16) + 2), dict(dS0=_addr(8) + 4), dict(dB=_heads(12, G, N, 8))):
        assert _scan_back(lib, **kw) == L.LQ_ERR_ALIGN, kw
    for kw in (dict(dx=_rows(1, CH)), dict(ddt=_rows(10, CH)), dict(dB=_heads(13, G, N)), dict(dz=_rows(6, CH)),
               dict(dA=_addr(20)), dict(dD=_addr(15) + 64), dict(db=_addr(16)), dict(dS0=_addr(7) + 64), dict(ws=_addr(12))):
        assert _scan_back(lib, **kw) == L.LQ_ERR_ALIAS, kw


@pytest.mark.parametrize("channels,groups", [(64, 1), (4096, 1), (1111, 11), (1 << 18, 2)])
def test_scan_workspace_covers_smaller_calls(lib, channels, groups):
    kw = dict(channels=channels, groups=groups)
    rows = dict(x=_rows(1, channels), dt=_rows(2, channels), z=None, B=_heads(3, groups, N), C=_heads(4, groups, N),
                y=_rows(1, channels))
    for save in (0, 1):
        size = lambda t, s: lib.leapquant_scan_workspace(_by(_sc(tokens=t, seqs=s, **kw)), save)  # noqa: E731
        for most in (1, 8, 9, 32, 33, 100, 700, 5000, 70000):
            for t in {1, 31, most // 3, most // 2, most - 1, most}:
                if 0 < t <= most:
                    for s in (1, 3):
                        # (y shares memory with x: refused behind the workspace's size)
                        ws = _addr(9) if size(most, 3) else None
                        assert _scan(lib, _sc(tokens=t, seqs=s, **kw), save, ws=ws, nbytes=size(most, 3), S0=None, S=None,
                                     **rows) == L.LQ_ERR_ALIAS, (most, t, s)
    assert lib.leapquant_scan_workspace(_by(_sc(tokens=8)), 0) == 0 < lib.leapquant_scan_workspace(_by(_sc(tokens=9)), 0)


# ---------------------------------------------------------------- block norm
H, DIM = 4, 128


def _bn(**kw):
    d = dict(tokens=T, heads=H, dim=DIM, dtype=L.LQ_BF16, dtype_stream=L.LQ_F32, gate=L.LQ_ACT_SILU, out_norm=1, eps=1e-6,
             scale=1.0, out_weight=_addr(20), in_weight=_addr(21))
    d.update(kw)
    return L.LqBlockNorm(*[d[f] for f, _ in L.LqBlockNorm._fields_])


def _norm(lib, bn=None, **kw):
    a = dict(a=_heads(1, H, DIM), z=_heads(2, H, DIM), res=_heads(3, H, DIM), h=_heads(4, H, DIM), y=_heads(5, H, DIM))
    a.update(kw)
    return lib.leapquant_block_norm(_by(bn or _bn()), *[_by(a[m]) for m in ("a", "z", "res", "h", "y")], None)


def _norm_back(lib, bn=None, **kw):
    a = dict(a=_heads(1, H, DIM), z=_heads(2, H, DIM), res=_heads(3, H, DIM), dh=_heads(4, H, DIM), dy=_heads(5, H, DIM),
             da=_heads(6, H, DIM), dz=_heads(7, H, DIM), dres=_heads(8, H, DIM), dwo=_addr(9), dwi=_addr(10), ws=_addr(11),
             nbytes=1 << 30)
    a.update(kw)
    r = [_by(a[m]) for m in ("a", "z", "res", "dh", "dy", "da", "dz", "dres")]
    return lib.leapquant_block_norm_backward(_by(bn or _bn()), *r, a["dwo"], a["dwi"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(heads=0), dict(heads=1 << 16), dict(dim=0),
                                dict(dim=12), dict(dim=8200), dict(dtype=3), dict(dtype_stream=-1), dict(gate=3),
                                dict(out_norm=2), dict(eps=0.0), dict(eps=float("nan")), dict(tokens=1 << 30)])
def test_block_norm_shapes(lib, kw):
    assert _norm(lib, _bn(**kw)) == L.LQ_ERR_SHAPE
    assert _norm_back(lib, _bn(**kw)) == L.LQ_ERR_SHAPE


def test_block_norm_refusals(lib):
    assert _norm(lib, _bn(dtype_stream=L.LQ_F16)) == L.LQ_ERR_UNSUPPORTED
    assert _norm(lib, _bn(dtype=L.LQ_F32, dtype_stream=L.LQ_BF16)) == L.LQ_ERR_UNSUPPORTED
    for kw in (dict(a=None), dict(z=None), dict(h=None, y=None), dict(res=L.LqRows(None, 512, 128))):
        assert _norm(lib, **kw) == L.LQ_ERR_NULL, kw
    assert _norm(lib, _bn(gate=L.LQ_ACT_NONE)) == L.LQ_ERR_SHAPE   # z without a gate
    assert _norm(lib, _bn(out_weight=_addr(20) + 4)) == L.LQ_ERR_ALIGN
    assert _norm(lib, a=_heads(1, H, DIM, 8)) == L.LQ_ERR_ALIGN
    assert _norm(lib, h=L.LqRows(_addr(4), 514, 128)) == L.LQ_ERR_ALIGN
    assert _norm(lib, y=L.LqRows(_addr(5), 0, 128)) == L.LQ_ERR_SHAPE
    for kw in (dict(y=_heads(2, H, DIM)), dict(h=_heads(1, H, DIM)), dict(y=_heads(4, H, DIM)), dict(y=_heads(20, H, DIM)),
               dict(h=L.LqRows(_addr(3), 1024, 128)), dict(y=L.LqRows(_addr(1) + 256, 512, 128))):
        assert _norm(lib, **kw) == L.LQ_ERR_ALIAS, kw


def test_block_norm_backward_refusals(lib):
    for kw in (dict(a=None), dict(z=None), dict(da=None), dict(dz=None), dict(dh=None, dy=None), dict(res=None),
               dict(dy=None), dict(ws=None)):
        assert _norm_back(lib, **kw) == L.LQ_ERR_NULL, kw
    assert _norm_back(lib, _bn(out_norm=0)) == L.LQ_ERR_SHAPE      # its weight's gradient
    assert _norm_back(lib, _bn(gate=L.LQ_ACT_NONE), z=None) == L.LQ_ERR_SHAPE
    assert _norm_back(lib, nbytes=100) == L.LQ_ERR_SHAPE
    assert _norm_back(lib, ws=_addr(11) + 4) == L.LQ_ERR_ALIGN
    assert _norm_back(lib, dwi=_addr(10) + 2) == L.LQ_ERR_ALIGN
    for kw in (dict(da=_heads(1, H, DIM)), dict(da=_heads(5, H, DIM)), dict(dz=_heads(6, H, DIM)),
               dict(dres=L.LqRows(_addr(4), 1024, 128)), dict(dres=_heads(3, H, DIM)), dict(dwo=_addr(20)),
               dict(dwi=_addr(9) + 64), dict(ws=_addr(8))):
        assert _norm_back(lib, **kw) == L.LQ_ERR_ALIAS, kw
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 7), (1, 1, 9000)):
        assert lib.leapquant_block_norm_workspace(*bad) == L.LQ_ERR_SHAPE
    assert lib.leapquant_block_norm_workspace(0, 1, 8) == 0 < lib.leapquant_block_norm_workspace(1, 1, 8)


# ---------------------------------------------------------------- the binding
def test_binding_refusals_without_a_device():
    x, w = torch.zeros(5, 8), torch.zeros(8, 4)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        lq.leapquant_conv_forward(cu, x, w, x)
    with pytest.raises(ValueError, match="2-D"):
        lq.leapquant_conv_forward(cu, x[None], w, x)
    with pytest.raises(ValueError, match="device memory|state on"):
        lq.leapquant_conv_step(x, w, x, torch.zeros(5, 3, 8))
    with pytest.raises(lq.LeapQuantError):
        lq.leapquant_conv_workspace(5, 1, 8, 7, device="cpu")
    with pytest.raises(lq.LeapQuantError):
        lq.LeapQuantScan(10, 1, 8, 5, device="cpu")
    with pytest.raises(lq.LeapQuantError):
        lq.LeapQuantScan(10, 1, 9, 8, groups=2, device="cpu")
    with pytest.raises(ValueError, match="dtype"):
        lq.LeapQuantScan(10, 1, 8, 8, dtype=torch.float64, device="cpu")
    plan = lq.LeapQuantScan(10, 1, 8, 8, dtype=torch.float32, device="cpu")
    A, b = torch.zeros(8, 8), torch.zeros(5, 1, 8)
    with pytest.raises(ValueError, match="device memory"):
        lq.leapquant_scan_forward(plan, cu, x, x, A, b, b, x)
    with pytest.raises(ValueError, match="without save"):
        lq.leapquant_scan_backward(plan, cu, x, x, A, b, b, x, x, x, A, b, b)
    saved = lq.LeapQuantScan(10, 1, 8, 8, dtype=torch.float32, device="cpu", save=True)
    with pytest.raises(ValueError, match="no forward"):
        lq.leapquant_scan_backward(saved, cu, x, x, A, b, b, x, x, x, A, b, b)
    a = torch.zeros(5, 1, 8)
    with pytest.raises(ValueError, match="h or y"):
        lq.leapquant_block_norm(a)
    with pytest.raises(ValueError, match="activation"):
        lq.leapquant_block_norm(a, h=a, z=a, gate="relu")
    with pytest.raises(ValueError, match="needs a gate"):
        lq.leapquant_block_norm(a, h=a, z=a, gate="none")
    with pytest.raises(ValueError, match="out_norm"):
        lq.leapquant_block_norm(a, h=a, out_weight=torch.zeros(8))
    with pytest.raises(ValueError, match="come together"):
        lq.leapquant_block_norm_backward(a, a, dh=a, z=a)
    with pytest.raises(ValueError, match="dres comes with res"):
        lq.leapquant_block_norm_backward(a, a, dh=a, dres=a)


STUB = r"""
#include <stdio.h>
#include <stdlib.h>
#include "lq_layer.h"
namespace lq {
static hipError_t reached() { fprintf(stderr, "launch reached\n"); abort(); }
hipError_t launch_conv(const ConvArgs &, int, bool, hipStream_t) { return reached(); }
hipError_t launch_conv_step(const ConvArgs &, int, bool, hipStream_t) { return reached(); }
hipError_t launch_conv_backward(const ConvArgs &, int, bool, hipStream_t) { return reached(); }
hipError_t launch_scan(const ScanArgs &, int, int, hipStream_t) { return reached(); }
hipError_t launch_scan_step(const ScanArgs &, int, int, hipStream_t) { return reached(); }
hipError_t launch_scan_backward(const ScanArgs &, int, int, hipStream_t) { return reached(); }
int64_t block_norm_blocks(int64_t, int) { return 7; }
hipError_t launch_block_norm(const BlockNormArgs &, int, int, hipStream_t) { return reached(); }
hipError_t launch_block_norm_backward(const BlockNormArgs &, int, int, hipStream_t) { return reached(); }
}  // namespace lq
#include "leapquant.h"
// extreme strides, sizes and addresses: each has to be refused without overflow
int main() {
  const int64_t strides[] = {0, 1, 127, 128, 512, int64_t(1) << 30, int64_t(1) << 46, INT64_MAX, INT64_MIN, -8};
  const int64_t toks[] = {1, 100, int64_t(1) << 30, INT64_MAX, INT64_MIN};
  const int sizes[] = {1, 8, 65535, 65536, 1 << 20, INT32_MAX, INT32_MIN};
  float *w = (float *)0x7f5000000000;
  const int32_t *cu = (const int32_t *)0x7f2000000000;
  int refused = 0, asked = 0;
  for (int64_t t : toks)
    for (int n : sizes)
      for (int m : sizes)
        for (int64_t a : strides) {
          lq_rows r = {(void *)0x7f0000000000, a, 16}, s = {(void *)0x7f1000000000, a, 16};
          // every output is the rows of an input: a call is refused at the latest for that
          lq_conv cv = {t, m, n, 4, LQ_ACT_SILU, LQ_F32, w, w};
          lq_scan sc = {t, m, n, 16, m, LQ_F32, 1u, w, w, w};
          lq_block_norm bn = {t, m, n, LQ_F32, LQ_F32, LQ_ACT_SILU, 1, 1e-6f, 1.f, w, w};
          const int rc[] = {
              leapquant_conv_forward(&cv, cu, &r, &r, w, nullptr, nullptr),
              leapquant_conv_step(&cv, cu, m, &r, &r, w, w, nullptr),
              leapquant_conv_backward(&cv, cu, &r, &s, &r, w, w, nullptr, nullptr, nullptr, nullptr, 0, nullptr),
              leapquant_scan_forward(&sc, cu, &r, &r, &s, &s, &r, &r, w, w, (void *)0x7f4000000000, INT64_MAX, 1, nullptr),
              leapquant_scan_step(&sc, cu, m, &r, &r, &s, &s, &r, &r, w, w, nullptr),
              leapquant_scan_backward(&sc, cu, &r, &r, &s, &s, &r, &r, &r, &r, &s, &s, &r, w, w, w, w, w,
                                      (void *)0x7f4000000000, INT64_MAX, nullptr),
              leapquant_block_norm(&bn, &r, &s, &r, &s, &s, nullptr),
              leapquant_block_norm_backward(&bn, &r, &s, &r, &s, &s, &r, &s, &s, nullptr, nullptr, nullptr, 0, nullptr)};
          for (int k : rc) ++asked, refused += k < 0;
          leapquant_conv_workspace(&cv);
          leapquant_scan_workspace(&sc, 1);
          leapquant_block_norm_workspace(t, m, n);
        }
  printf("%d of %d refused\n", refused, asked);
  return refused == asked ? 0 : 1;
}
"""


def test_argument_checks_under_asan_and_ubsan(tmp_path):
    from tests.test_sanitizers import ROCM, ROOT, SAN, _run
    src = tmp_path / "driver.cpp"
    src.write_text(STUB)
    inc = ["-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "recurrent_state_quant_amd", "csrc"), "-I", os.path.join(ROCM, "include")]
    exe = tmp_path / "driver"
    _run(["g++", "-std=c++17", "-O1", *SAN, *inc, "-o", str(exe), str(src),
          os.path.join(ROOT, "recurrent_state_quant_amd", "csrc", "lq_layer_abi.cpp")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    res = _run([str(exe)], env=env, timeout=120)
    assert "refused" in res.stdout


@pytest.mark.parametrize("std", ["c99", "c11"])
def test_refusals_from_c(tmp_path, std):
    from tests.test_c_abi import ROCM, ROOT
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libleapquant.so is not built (run __graft_entry__.build())")
    exe = str(tmp_path / "checks")
    res = subprocess.run(["gcc", f"-std={std}", "-O2", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"), "-o", exe,
                          os.path.join(ROOT, "tests", "c_abi", "lq_layer_checks.c"), "-L", os.path.dirname(B.LIB_PATH),
                          "-lleapquant", "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                          f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "layer checks passed" in res.stdout
