"""Blockwise codes of the norm are those of a division, whatever the scale.

tests/e4m3_quotient_fp32_check.c walks every pair of fp32 value and scale at
which the kernel's corrected product could give another code than the fp32
quotient, from the smallest scale that the kernel uses it for (norm.cu's
kQuotientMin)."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixture_experts_layer_sigmoid_gb300", "csrc")


def test_corrected_product_gives_the_divisions_codes(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = open(os.path.join(CSRC, "norm.cu")).read()
    border = re.search(r"constexpr float kQuotientMin = 0x1p(-\d+)f", src)
    assert border, "norm.cu: kQuotientMin"
    exe = str(tmp_path / "check")
    subprocess.run([cc, "-O2", "-ffp-contract=off", "-o", exe, os.path.join(HERE, "e4m3_quotient_fp32_check.c"), "-lm"],
                   check=True)
    r = subprocess.run([exe, border.group(1)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "E4M3 differences 0" in r.stdout, r.stdout
