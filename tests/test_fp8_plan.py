"""Which kernel the 8-bit floating point product takes (csrc/fp8_plan.hpp, compiled
for the host; no GPU needed): what the estimate of the time is for is what is
launched, whatever the table of tokens holds, and the shapes that the GPU tests use
reach the kernels that they are there for."""
import os
import subprocess

import pytest

from tests.test_gpu_block_plans import SHAPES
from tests.test_gpu_block_tables import PRODUCTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "fp8_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "communication_efficient_gradient_amd", "csrc"),
                    os.path.join(ROOT, "tests", "fp8_plan.cpp"), "-o", out], check=True)
    return out


def test_any_table_fits_the_plan(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    said = r.stdout.split()
    assert said[0] == "ok" and all(int(n) > 1000 for n in said[1:])


def test_shapes_reach_their_kernels(exe):
    for kernel, shapes in [*SHAPES.items(), *PRODUCTS.items()]:
        for rows, out, cols, experts in shapes:
            k_tiles = -(-cols // 128)
            r = subprocess.run([exe, *map(str, (rows, k_tiles, out, experts))],
                               capture_output=True, text=True, timeout=60, check=True)
            tile, teams, splits, per, _ = map(int, r.stdout.split())
            got = (tile, teams, "parts" if splits > 1 else "whole", "odd" if per % 2 else "even")
            assert kernel == got[:len(kernel)], (rows, out, cols, experts)


def test_few_tokens_of_several_experts_by_what_was_measured(exe):
    """Tokens, k-tiles, out, experts: the kernel that measured faster by more than a
    quarter with even and with uneven loads."""
    few = [(32, 16, 1024, 16), (8, 32, 1024, 4), (32, 33, 2050, 2), (64, 33, 2050, 16),
           (24, 12, 512, 48)]
    tiled = [(64, 32, 4096, 2), (48, 64, 8192, 2), (64, 64, 4608, 2), (60, 40, 5120, 3),
             (64, 32, 14336, 2), (64, 8, 4096, 64), (60, 10, 12000, 48)]
    for shape in few + tiled:
        r = subprocess.run([exe, *map(str, shape)], capture_output=True, text=True, timeout=60,
                           check=True)
        assert (r.stdout.split()[0] == "0") == (shape in few), shape
