"""Index bounds of the 8-bit activation kernels, on the CPU: the loads of the
weight gradient's way through registers stay inside dy.  The bounds are plain
C++ that the library shares (csrc/act_bounds.hpp)."""
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


def test_loads_stay_inside(walk):
    r = subprocess.run([walk], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
