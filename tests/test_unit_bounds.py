"""What the weight gradient by expert launches and keeps in its workspace holds
every table's units and parts (csrc/act_bounds.hpp, compiled for the host; no GPU
needed)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_units_and_parts(tmp_path):
    exe = str(tmp_path / "unit_bounds")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "communication_efficient_gradient_amd", "csrc"),
                    os.path.join(ROOT, "tests", "unit_bounds.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ok ")
