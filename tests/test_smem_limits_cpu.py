"""The table of shared-memory limits that launches consult (host code)."""
import os
import subprocess

from conftest import ROOT


def test_limits_only_rise(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "ternary_weight_linear_absmax_b200", "csrc"),
                    os.path.join(ROOT, "tests", "smem_limits_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
