"""The rules by which calls of the convolution are cut into runs (csrc/lq_layer.h;
CPU)."""
import ctypes
import os
import subprocess

import pytest

SOURCE = r"""
#include "lq_layer.h"
using namespace lq;
extern "C" {
int run_tokens(int64_t t, int64_t tiles, int least) { return conv_run_tokens(t, tiles, least); }
int grad_run(int64_t t, int64_t c) { return conv_grad_run(t, c); }
int64_t grad_blocks(int64_t t, int64_t run) { return conv_grad_blocks(t, run); }
int64_t most_blocks(int64_t t) { return conv_grad_most(t); }
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
    for name, args, back in (("run_tokens", [i64, i64, i32], i32), ("grad_run", [i64, i64], i32),
                             ("grad_blocks", [i64, i64], i64), ("most_blocks", [i64], i64)):
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
