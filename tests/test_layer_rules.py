"""The rules by which calls of the convolution and the scan are cut into runs and
chunks (csrc/lq_layer.h), and the 64-bit forms of the larger tests (CPU)."""
import ctypes
import os
import subprocess

import pytest
import torch

from tests import layer_reference as R
from tests import scan_beside

SOURCE = r"""
#include "lq_layer.h"
using namespace lq;
extern "C" {
int forward_chunk(int64_t t, int64_t s, int c, int g, int n) { return scan_forward_chunk(t, s, c, g, n); }
int grad_chunk(int64_t t, int64_t s, int c, int g, int n) { return scan_grad_chunk(t, s, c, g, n); }
int grad_part(int chunk) { return scan_grad_part(chunk); }
int run_tokens(int64_t t, int64_t tiles, int least) { return conv_run_tokens(t, tiles, least); }
int grad_run(int64_t t, int64_t c) { return conv_grad_run(t, c); }
int64_t grad_blocks(int64_t t, int64_t run) { return conv_grad_blocks(t, run); }
int64_t most_blocks(int64_t t) { return conv_grad_most(t); }
int64_t slots(int64_t t, int64_t s, int chunk) { return scan_slots(t, s, chunk); }
int64_t most_chunks(int64_t t, int64_t s, int c, int g, int n) { return scan_most_chunks(t, s, c, g, n); }
int64_t most_slots(int64_t t, int64_t s, int c, int g, int n, int grad) { return scan_most_slots(t, s, c, g, n, grad); }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    from tests.test_sanitizers import ROCM, ROOT
    d = tmp_path_factory.mktemp("rules")
    src, out = d / "rules.cpp", d / "rules.so"
    src.write_text(SOURCE)
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I",
                          os.path.join(ROOT, "recurrent_state_quant_amd", "csrc"), "-I", os.path.join(ROCM, "include"),
                          "-o", str(out), str(src)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    lib = ctypes.CDLL(str(out))
    i64, i32 = ctypes.c_int64, ctypes.c_int
    scan = [i64, i64, i32, i32, i32]
    for name, args, back in (("forward_chunk", scan, i32), ("grad_chunk", scan, i32), ("grad_part", [i32], i32),
                             ("run_tokens", [i64, i64, i32], i32), ("grad_run", [i64, i64], i32),
                             ("grad_blocks", [i64, i64], i64), ("most_blocks", [i64], i64), ("slots", [i64, i64, i32], i64),
                             ("most_slots", scan + [i32], i64), ("most_chunks", scan, i64)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, back
    return lib


def test_runs_that_the_gpu_tests_mean(rules):
    from tests.test_gpu_conv_sums import CASES, F32
    for tokens, c, dtype, run, run_grad, blocks in CASES:
        tile = 64 * (4 if dtype == F32 else 8)   # channels of a wave: 16 bytes a lane
        assert rules.run_tokens(tokens, -(-c // tile), 4) == run
        assert rules.grad_run(tokens, c) == run_grad and rules.grad_blocks(tokens, run_grad) == blocks
        assert blocks <= rules.most_blocks(tokens)


def test_chunks_that_the_gpu_tests_mean(rules):
    from tests.test_gpu_scan_chunks import CHANNELS, CHUNKS, CU, TOKENS
    for states, (forward, grad) in CHUNKS.items():
        for groups in (1, 2):
            args = TOKENS, len(CU) - 1, CHANNELS, groups, states
            assert rules.forward_chunk(*args) == forward >= 32 and rules.grad_chunk(*args) == grad >= 32
            part = rules.grad_part(grad)
            assert part == grad // 2
            for chunk in (forward, grad, part):
                # several a sequence, whose last one ends inside the tokens that are loaded together, eight or four
                lens = [b - a for a, b in zip(CU, CU[1:])]
                assert sum(m > 2 * chunk for m in lens) == 2 and all(m % chunk % 4 for m in lens if m > chunk)


SIZES = [0, 1, 7, 8, 9, 31, 32, 33, 63, 100, 250, 511, 512, 513, 1021, 4096, 5000, 16384, 70001, 1 << 20, 1 << 26]


@pytest.mark.parametrize("states", [8, 16, 32])
def test_chunks_fit_the_workspace(rules, states):
    """Every chunk length is one that the kernels and the workspace are made for, and a call with fewer tokens or
    sequences needs no more slots."""
    for channels, groups in ((1, 1), (64, 1), (1111, 11), (2048, 1), (4096, 4), (1 << 16, 2), (1 << 20, 1)):
        last = {}
        for tokens in SIZES:
            for seqs in (1, 2, 5, 24, 1000, 100_000):
                args = tokens, seqs, channels, groups, states
                forward, grad = rules.forward_chunk(*args), rules.grad_chunk(*args)
                part = rules.grad_part(grad)
                for chunk in (forward, grad):
                    assert chunk % 8 == 0 and 8 <= chunk <= 512
                assert part % 4 == 0 and grad % part == 0 and grad // part <= 2
                if tokens <= 8:
                    assert forward >= tokens   # one chunk: a forward call needs no workspace
                only, both, whole = rules.most_slots(*args, 0), rules.most_slots(*args, 1), rules.most_chunks(*args)
                assert rules.slots(tokens, seqs, forward) <= only <= both and rules.slots(tokens, seqs, part) <= both
                assert rules.slots(tokens, seqs, grad) <= whole <= both
                for smaller in (v for k, v in last.items() if k[0] <= tokens and k[1] <= seqs):
                    assert smaller[0] <= only and smaller[1] <= both and smaller[2] <= whole
                last[tokens, seqs] = only, both, whole


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("plain", [True, False])
def test_sequences_beside_one_another(softplus, plain):
    """The 64-bit scan of the larger tests is the one of the others."""
    g = torch.Generator().manual_seed(5)
    cu, T, c, N, G = [1, 6, 6, 19, 20], 22, 6, 3, 2
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    v = [r(T, c), r(T, c), -torch.rand((c, N), generator=g, dtype=torch.float64), r(T, G, N), r(T, G, N), r(c), r(c), r(T, c),
         r(4, c, N), r(T, c), r(4, c, N)]
    if plain:
        v[5] = v[6] = v[7] = None
    for absolute in (False, True):
        a, b = (f.scan_adjoint(cu, *v, softplus=softplus, absolute=absolute) for f in (R, scan_beside))
        assert set(a) - {"D"} <= set(b)
        for m in b:
            if m == "z" and absolute:   # (there by the slope's own value)
                assert (b[m] >= a[m] * (1 - 1e-12)).all()
            else:
                assert torch.allclose(a[m], b[m], rtol=1e-10, atol=1e-12), m


def test_workspace_of_a_training_step():
    """8,192 tokens in 4 sequences, 2,048 channels, 16 states: states kept before every fourth token, states carried and
    steps summed for chunks from zero of at least 16 tokens, shares of dB and dC of every wave of 64 channels, shares of
    dA, dD and dbias for chunks of at least 32 tokens."""
    import recurrent_state_quant_amd as lq
    T, seqs, c, N = 8192, 4, 2048, 16
    plan = lq.LeapQuantScan(T, seqs, c, N, device="cpu", save=True)
    parts, chunks = T // 16 + seqs, T // 32 + seqs
    kept, carried, sums = (T // 4 + seqs) * c * N * 4, parts * c * N * 4, parts * c * 4
    shares, weights = c // 64 * T * 2 * N * 4, chunks * (N + 2) * c * 4
    assert plan.workspace.numel() == kept + carried + sums + shares + weights
    assert [round(v / 1e6) for v in (kept, carried, sums, shares, weights)] == [269, 68, 4, 34, 38]
