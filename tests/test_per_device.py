"""Answers of device queries are kept per device, and failed queries are not (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_grouped_align_gb300", "csrc")


def test_per_device_table(tmp_path):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "per_device_check")
    r = subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(ROOT, "tests", "c", "per_device_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_dense_plan_s_queries_go_through_it():
    """No table of the plan is indexed by anything but the device."""
    text = open(os.path.join(CSRC, "dense_split.cu")).read()
    assert "PerDevice<9>" in text and "std::atomic<int> seen" not in text
