"""What the first call of a kernel on a device keeps: csrc/per_device.h, on the host."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixture_experts_layer_sigmoid_gb300", "csrc")


def test_an_error_is_not_kept(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "per_device_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", exe, os.path.join(HERE, "per_device_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_products_keep_nothing_else():
    """No value of a first call in a function's static of its own (one would hold an error, and for every device)."""
    for f in ("grouped_tc.cuh", "grouped_tc_rows.cu", "grouped_tc_wgrad.cu", "grouped_simt.cu", "matmul_fp8.cu", "products.cu"):
        for line in open(os.path.join(CSRC, f)):
            assert "static const cudaError_t" not in line and "once_flag" not in line, (f, line)
