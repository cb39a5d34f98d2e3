"""Refusals of the sequence entry points (CPU): every call here is rejected by
host-side validation before any launch, so fake addresses are safe; and the
same checks under AddressSanitizer and UBSan are in the last test."""
import ctypes

import pytest
import torch

import recurrent_state_quant_amd as lq
from recurrent_state_quant_amd import _lib as L

BASE = 0x7F0000000000  # never dereferenced
MB = 1 << 20
T, SEQS, HK, HV = 100, 3, 2, 4


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _sq(**kw):
    d = dict(tokens=T, seqs=SEQS, heads_k=HK, heads_v=HV, dk=128, dv=128, gate=L.LQ_GATE_GDN, flags=0, dtype=L.LQ_BF16)
    d.update(kw)
    return L.LqSequence(*[d[f] for f, _ in L.LqSequence._fields_])


def _addr(i):
    return BASE + i * 64 * MB


def _rows(i, heads, width=128, off=0):
    return L.LqRows(_addr(i) + off, heads * width, width)


def _forward(lib, sq=None, save=0, **kw):
    a = dict(cu=_addr(0), q=_rows(1, HK), k=_rows(2, HK), v=_rows(3, HV), beta=_rows(4, HV, 1), alpha=_rows(5, HV, 1),
             o=_rows(6, HV), S0=_addr(7), S=_addr(8), ws=_addr(9), nbytes=1 << 40)
    a.update(kw)
    r = [None if a[x] is None else ctypes.byref(a[x]) for x in ("q", "k", "v", "beta", "alpha", "o")]
    return lib.leapquant_sequence_forward(ctypes.byref(sq or _sq()), a["cu"], *r, a["S0"], a["S"], a["ws"],
                                          a["nbytes"], save, None)


def _backward(lib, sq=None, **kw):
    a = dict(cu=_addr(0), q=_rows(1, HK), k=_rows(2, HK), beta=_rows(4, HV, 1), alpha=_rows(5, HV, 1), go=_rows(6, HV),
             dS=_addr(7), dq=_rows(10, HK), dk=_rows(11, HK), dv=_rows(12, HV), dbeta=_rows(13, HV, 1),
             dalpha=_rows(14, HV, 1), dS0=_addr(8), ws=_addr(9), nbytes=1 << 40)
    a.update(kw)
    r = {x: None if a[x] is None else ctypes.byref(a[x]) for x in
         ("q", "k", "beta", "alpha", "go", "dq", "dk", "dv", "dbeta", "dalpha")}
    return lib.leapquant_sequence_backward(ctypes.byref(sq or _sq()), a["cu"], r["q"], r["k"], r["beta"], r["alpha"],
                                           r["go"], a["dS"], r["dq"], r["dk"], r["dv"], r["dbeta"], r["dalpha"],
                                           a["dS0"], a["ws"], a["nbytes"], None)


SHAPES = [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(seqs=0), dict(seqs=1 << 24), dict(heads_k=0),
          dict(heads_k=3), dict(heads_v=0), dict(heads_v=1 << 17, heads_k=1), dict(gate=2), dict(flags=1), dict(dtype=3),
          dict(flags=L.LQ_NO_DELTA | 8)]


@pytest.mark.parametrize("kw", SHAPES)
def test_sequence_shapes(lib, kw):
    sq = _sq(**kw)
    assert _forward(lib, sq) == L.LQ_ERR_SHAPE
    assert _backward(lib, sq) == L.LQ_ERR_SHAPE
    assert lib.leapquant_sequence_workspace(ctypes.byref(sq), 0) == L.LQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [dict(dk=64), dict(dv=256)])
def test_sequence_head_size(lib, kw):
    assert _forward(lib, _sq(**kw)) == L.LQ_ERR_UNSUPPORTED
    assert _backward(lib, _sq(**kw)) == L.LQ_ERR_UNSUPPORTED


def test_per_channel_gate_has_no_backward(lib):
    sq = _sq(gate=L.LQ_GATE_KDA)
    assert _forward(lib, sq, save=1) == L.LQ_ERR_UNSUPPORTED
    assert _backward(lib, sq) == L.LQ_ERR_UNSUPPORTED
    assert lib.leapquant_sequence_workspace(ctypes.byref(sq), 1) == L.LQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["cu", "q", "k", "v", "beta", "alpha", "o", "ws"])
def test_forward_null(lib, name):
    assert _forward(lib, **{name: None}) == L.LQ_ERR_NULL
    if name not in ("cu", "ws"):
        assert _forward(lib, **{name: L.LqRows(None, 512, 128)}) == L.LQ_ERR_NULL


@pytest.mark.parametrize("name", ["cu", "q", "k", "beta", "alpha", "go", "dq", "dk", "dv", "dbeta", "dalpha", "ws"])
def test_backward_null(lib, name):
    assert _backward(lib, **{name: None}) == L.LQ_ERR_NULL


@pytest.mark.parametrize("kw", [dict(q=_rows(1, HK, off=8)), dict(o=_rows(6, HV, off=2)), dict(beta=_rows(4, HV, 1, 2)),
                                dict(S0=_addr(7) + 4), dict(S=_addr(8) + 8), dict(cu=_addr(0) + 2),
                                dict(ws=_addr(9) + 4), dict(k=L.LqRows(_addr(2), 260, 128)),
                                dict(v=L.LqRows(_addr(3), 512, 132))])
def test_forward_alignment(lib, kw):
    assert _forward(lib, **kw) == L.LQ_ERR_ALIGN


@pytest.mark.parametrize("kw", [dict(q=L.LqRows(_addr(1), -256, 128)), dict(v=L.LqRows(_addr(3), 1 << 50, 128)),
                                dict(o=L.LqRows(_addr(6), 0, 128)), dict(o=L.LqRows(_addr(6), 512, 64)),
                                dict(o=L.LqRows(_addr(6), 128, 128)), dict(nbytes=1000)])
def test_forward_strides_and_workspace(lib, kw):
    assert _forward(lib, **kw) == L.LQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [
    dict(o=_rows(1, HV)), dict(o=_rows(3, HV)), dict(S=_addr(3)), dict(S=_addr(7) + 256), dict(ws=_addr(2)),
    dict(ws=_addr(0)), dict(S=_addr(6)), dict(o=_rows(4, HV)), dict(S=_addr(0)),
    # one row of o reaches into v's rows of the same pitch
    dict(v=L.LqRows(_addr(6) + 2 * 256, 1024, 128), o=L.LqRows(_addr(6), 1024, 128))])
def test_forward_overlap(lib, kw):
    assert _forward(lib, **kw) == L.LQ_ERR_ALIAS


@pytest.mark.parametrize("kw", [dict(dq=_rows(1, HK)), dict(dk=_rows(10, HK)), dict(dv=_rows(6, HV)),
                                dict(dbeta=_rows(14, HV, 1)), dict(dalpha=_rows(5, HV, 1)), dict(dS0=_addr(7) + 512),
                                dict(ws=_addr(12)), dict(dS0=_addr(9)),
                                # gradients interleaved in one row, one of them too wide
                                dict(dq=L.LqRows(_addr(10), 768, 128), dk=L.LqRows(_addr(10) + 256, 768, 128))])
def test_backward_overlap(lib, kw):
    assert _backward(lib, **kw) == L.LQ_ERR_ALIAS


def test_workspace_covers_smaller_calls(lib):
    size = lambda **kw: lib.leapquant_sequence_workspace(ctypes.byref(_sq(**kw)), 0)  # noqa: E731
    most = size(tokens=1000, seqs=50)
    for tokens in (0, 1, 16, 17, 500, 999, 1000):
        for seqs in (1, 2, 30, 50):
            assert 0 <= size(tokens=tokens, seqs=seqs) <= most
            need = ctypes.c_int64(most)
            # a null output is refused after the workspace's size is: the size is enough
            assert _forward(lib, _sq(tokens=tokens, seqs=seqs), nbytes=need.value,
                            o=None) == L.LQ_ERR_NULL
    assert size(tokens=10, seqs=5) == 0
    assert size(gate=L.LQ_GATE_KDA, tokens=10) == 0 < size(gate=L.LQ_GATE_KDA, tokens=1000)
    assert lib.leapquant_sequence_workspace(ctypes.byref(_sq(tokens=10)), 1) > 0


def _nm(**kw):
    d = dict(tokens=T, heads_q=4, heads_k=2, dim=128, kind=0, dtype=L.LQ_BF16, dtype_out=L.LQ_F32, rot=64,
             interleaved=0, eps=1e-6, q_scale=1.0, q_weight=_addr(0), k_weight=_addr(0) + 4096, positions=_addr(1),
             inv_freq=_addr(2))
    d.update(kw)
    return L.LqHeadNorm(*[d[f] for f, _ in L.LqHeadNorm._fields_])


def _norm(lib, nm=None, **kw):
    a = dict(q=_rows(3, 4), k=_rows(4, 2), qo=_rows(5, 4), ko=_rows(6, 2))
    a.update(kw)
    r = [None if a[x] is None else ctypes.byref(a[x]) for x in ("q", "k", "qo", "ko")]
    return lib.leapquant_head_norm(ctypes.byref(nm or _nm()), *r, None)


def _norm_back(lib, nm=None, **kw):
    a = dict(q=_rows(3, 4), k=_rows(4, 2), gq=_rows(5, 4), gk=_rows(6, 2), dq=_rows(7, 4), dk=_rows(8, 2), dwq=_addr(9),
             dwk=_addr(9) + 4096, ws=_addr(10), nbytes=1 << 30)
    a.update(kw)
    r = [None if a[x] is None else ctypes.byref(a[x]) for x in ("q", "k", "gq", "gk", "dq", "dk")]
    return lib.leapquant_head_norm_backward(ctypes.byref(nm or _nm()), *r, a["dwq"], a["dwk"], a["ws"], a["nbytes"],
                                            None)


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(heads_q=-1), dict(heads_q=0, heads_k=0),
                                dict(heads_k=1 << 16), dict(kind=2), dict(dtype=5), dict(dtype_out=-1), dict(rot=8),
                                dict(rot=144), dict(rot=-16), dict(interleaved=2), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(tokens=1 << 30)])
def test_norm_shapes(lib, kw):
    assert _norm(lib, _nm(**kw)) == L.LQ_ERR_SHAPE
    assert _norm_back(lib, _nm(**kw)) == L.LQ_ERR_SHAPE


def test_norm_other_refusals(lib):
    assert _norm(lib, _nm(dim=64)) == L.LQ_ERR_UNSUPPORTED
    assert _norm(lib, _nm(positions=None)) == L.LQ_ERR_NULL
    assert _norm(lib, _nm(inv_freq=None)) == L.LQ_ERR_NULL
    for x in ("q", "k", "qo", "ko"):
        assert _norm(lib, **{x: None}) == L.LQ_ERR_NULL
        assert _norm(lib, **{x: L.LqRows(None, 512, 128)}) == L.LQ_ERR_NULL
    assert _norm(lib, _nm(positions=_addr(1) + 4)) == L.LQ_ERR_ALIGN
    assert _norm(lib, _nm(q_weight=_addr(0) + 2)) == L.LQ_ERR_ALIGN
    assert _norm(lib, q=_rows(3, 4, off=4)) == L.LQ_ERR_ALIGN
    assert _norm(lib, qo=L.LqRows(_addr(5), 0, 128)) == L.LQ_ERR_SHAPE
    # over its own input only in the same type and strides
    assert _norm(lib, qo=_rows(3, 4)) == L.LQ_ERR_ALIAS
    assert _norm(lib, _nm(dtype_out=L.LQ_BF16), qo=L.LqRows(_addr(3), 1024, 128)) == L.LQ_ERR_ALIAS
    assert _norm(lib, _nm(dtype_out=L.LQ_BF16), qo=_rows(4, 4)) == L.LQ_ERR_ALIAS
    assert _norm(lib, ko=_rows(5, 2)) == L.LQ_ERR_ALIAS
    assert _norm(lib, ko=_rows(1, 2)) == L.LQ_ERR_ALIAS


def test_norm_backward_refusals(lib):
    for x in ("q", "k", "gq", "gk", "dq", "dk", "ws"):
        assert _norm_back(lib, **{x: None}) == L.LQ_ERR_NULL
    assert _norm_back(lib, nbytes=100) == L.LQ_ERR_SHAPE
    assert _norm_back(lib, ws=_addr(10) + 8) == L.LQ_ERR_ALIGN
    assert _norm_back(lib, dwq=_addr(9) + 2) == L.LQ_ERR_ALIGN
    assert _norm_back(lib, dq=_rows(3, 4)) == L.LQ_ERR_ALIAS
    assert _norm_back(lib, dwk=_addr(9) + 256) == L.LQ_ERR_ALIAS
    assert _norm_back(lib, dwq=_addr(0)) == L.LQ_ERR_ALIAS
    assert _norm_back(lib, ws=_addr(8)) == L.LQ_ERR_ALIAS
    assert lib.leapquant_head_norm_workspace(-1, 1, 1) == L.LQ_ERR_SHAPE
    assert lib.leapquant_head_norm_workspace(5, 0, 0) == L.LQ_ERR_SHAPE
    assert lib.leapquant_head_norm_workspace(5, 4, 2) > 0


def test_binding_refusals_without_a_device():
    with pytest.raises(ValueError, match="dtype"):
        lq.LeapQuantSequence(10, 1, 1, 1, dtype=torch.float64, device="cpu")
    with pytest.raises(lq.LeapQuantError):
        lq.LeapQuantSequence(10, 1, 2, 3, device="cpu")
    with pytest.raises(lq.LeapQuantError):
        lq.LeapQuantSequence(10, 1, 1, 1, gate="kda", device="cpu", save=True)
    plan = lq.LeapQuantSequence(10, 2, 1, 1, dtype=torch.float32, device="cpu")
    x = torch.zeros(10, 1, 128)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        lq.leapquant_sequence_forward(plan, cu, x, x, x, x[..., 0], x[..., 0], x)
    with pytest.raises(ValueError, match="plan is for"):
        lq.leapquant_sequence_forward(plan, cu, torch.zeros(11, 1, 128), x, x, x, x, x)
    with pytest.raises(ValueError, match="without save"):
        lq.leapquant_sequence_backward(plan, cu, x, x, x, x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="come together"):
        lq.leapquant_head_norm(x, x, x, x, positions=cu)
    with pytest.raises(ValueError, match="unknown norm"):
        lq.leapquant_head_norm(x, x, x, x, norm="layer")


STUB = r"""
#include <stdio.h>
#include <stdlib.h>
#include "lq_sequence.h"
namespace lq {
static hipError_t reached() { fprintf(stderr, "launch reached\n"); abort(); }
hipError_t launch_seq_recurrent(const SeqArgs &, int, bool, bool, hipStream_t) { return reached(); }
hipError_t launch_seq_chunked(const SeqArgs &, int, bool, bool, hipStream_t) { return reached(); }
hipError_t launch_seq_backward(const SeqArgs &, int, bool, hipStream_t) { return reached(); }
int64_t norm_blocks(int64_t, int, int) { return 7; }
hipError_t launch_norm(const NormArgs &, int, int, hipStream_t) { return reached(); }
hipError_t launch_norm_backward(const NormArgs &, int, int, hipStream_t) { return reached(); }
}  // namespace lq
#include "leapquant.h"
// extreme strides, sizes and addresses: each has to be refused without overflow
int main() {
  const int64_t big[] = {0, 1, 127, 128, 512, int64_t(1) << 30, int64_t(1) << 46, INT64_MAX, INT64_MIN, -8};
  const int64_t toks[] = {0, 1, 100, int64_t(1) << 30, INT64_MAX, INT64_MIN};
  const int heads[] = {1, 2, 65535, 65536, INT32_MAX, INT32_MIN};
  int refused = 0, asked = 0;
  for (int64_t t : toks)
    for (int h : heads)
      for (int64_t a : big)
        for (int64_t b : big) {
          lq_sequence sq = {t, h, 1, h, 128, 128, 0, 0, 1};
          lq_rows r = {(void *)0x7f0000000000, a, b}, sc = {(void *)0x7f1000000000, a, b};
          // o is the rows of q: every call is refused at the latest for that
          const int rc = leapquant_sequence_forward(&sq, (const int32_t *)0x7f2000000000, &r, &r, &r, &sc, &sc, &r,
                                                    (const float *)0x7f3000000000, (float *)0x7f3000000010,
                                                    (void *)0x7f4000000000, INT64_MAX, 1, nullptr);
          lq_head_norm nm = {t, h, 1, 128, 0, 1, 1, 0, 0, 1e-6f, 1.f, nullptr, nullptr, nullptr, nullptr};
          const int rn = t == 0 ? -1 : leapquant_head_norm_backward(&nm, &r, &r, &r, &r, &r, &r, nullptr, nullptr, nullptr, 0, nullptr);
          ++asked;
          refused += rc < 0 && rn < 0;
        }
  printf("%d of %d refused\n", refused, asked);
  return refused == asked ? 0 : 1;
}
"""


def test_argument_checks_under_asan_and_ubsan(tmp_path):
    from tests.test_sanitizers import ROCM, ROOT, SAN, _run
    import os
    src = tmp_path / "driver.cpp"
    src.write_text(STUB)
    inc = ["-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "recurrent_state_quant_amd", "csrc"), "-I", os.path.join(ROCM, "include")]
    exe = tmp_path / "driver"
    _run(["g++", "-std=c++17", "-O1", *SAN, *inc, "-o", str(exe), str(src),
          os.path.join(ROOT, "recurrent_state_quant_amd", "csrc", "lq_sequence_abi.cpp")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    res = _run([str(exe)], env=env, timeout=120)
    assert "refused" in res.stdout
