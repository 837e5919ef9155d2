"""Index arithmetic of the 8-bit activation kernels, on the CPU: the loads of the
weight gradient's way through registers stay inside dy, and packing and
unpacking reach every value of the largest matrices in launches that the device
takes.  The rules are plain C++ that the library shares (csrc/act_bounds.hpp)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "communication_efficient_gradient_amd", "csrc")


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("bounds") / "act_bounds")
    cxx = shutil.which("g++") or shutil.which("clang++")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", f"-I{CSRC}",
                    os.path.join(HERE, "act_bounds.cpp"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("what", ["loads", "cover"])
def test_walk(walk, what):
    r = subprocess.run([walk, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
