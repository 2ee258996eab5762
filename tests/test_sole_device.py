"""Loads that a cluster shares (TMA multicast) belong to runs on one GPU alone (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_grouped_align_gb300", "csrc")


def test_sole_device(tmp_path):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "sole_device_check")
    r = subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, os.path.join(ROOT, "tests", "c", "sole_device_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_every_launch_with_shared_loads_asks():
    """The weight gradient's clusters are the only ones whose loads are multicast, and each launch of them is
    behind the question."""
    users = [f for f in sorted(os.listdir(CSRC)) if re.search(r"tma::load_2d_multicast", open(os.path.join(CSRC, f)).read())]
    assert users == ["wgrad_tc.cu"]
    text = open(os.path.join(CSRC, "wgrad_tc.cu")).read()
    launches = re.findall(r"if \(([^\n]*)\) \{\n\s*cudaError_t err = launch_slot<(\d)>", text)
    assert [c for _, c in launches] == ["4", "2"] and all(cond.startswith("alone && ") for cond, _ in launches)
    assert len(re.findall(r"launch_slot<[^1C]>", text)) == 2
    assert "const bool alone = moe_host::sole_device(" in text
