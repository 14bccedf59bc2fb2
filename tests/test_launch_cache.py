"""csrc/launch.cuh on the host alone: tests/c/launch_cache.cpp stands in for the
CUDA runtime and counts its calls (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from matrix_optimizers_zero_gb300 import build as mo_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_kernel_is_set_up_once(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(mo_build._nvcc()))), "include")
    exe = str(tmp_path / "launch_cache")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", cuda_inc, "-I", mo_build.CSRC, os.path.join(ROOT, "tests", "c", "launch_cache.cpp"),
                    "-o", exe, "-lpthread"], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
