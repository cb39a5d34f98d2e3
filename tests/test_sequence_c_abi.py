"""The sequence and head norm entry points from plain C (CPU)."""
import os
import subprocess

import pytest

from recurrent_state_quant_amd import build as B
from tests.test_c_abi import ROCM, ROOT


@pytest.mark.parametrize("std", ["c99", "c11"])
def test_refusals_from_c(tmp_path, std):
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libleapquant.so is not built (run __graft_entry__.build())")
    exe = str(tmp_path / "checks")
    res = subprocess.run(["gcc", f"-std={std}", "-O2", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
                          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"), "-o", exe,
                          os.path.join(ROOT, "tests", "c_abi", "lq_sequence_checks.c"), "-L", os.path.dirname(B.LIB_PATH),
                          "-lleapquant", "-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                          f"-Wl,-rpath,{os.path.dirname(B.LIB_PATH)}", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "sequence checks passed" in res.stdout
