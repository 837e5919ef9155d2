"""The weight gradients of matrices without rows, whose row pointer is NULL and
whose stride is whatever the caller has: a call of a program that sees no GPU ends
with a status (no GPU needed)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALL = """
from communication_efficient_gradient_amd import gq
L, M = gq.lib(), 1 << 24
a = gq.gq_act(0, 100, {dtype}, {group})
for ld in (0, 7, -5):
    if "{name}" == "gq_act_wgrad":
        rc = L.gq_act_wgrad(a, 50, None, ld, None, None, 0.0, M, 2 * M, None, 0, None)
    else:
        rc = L.gq_block_wgrad(a, 50, 1, None, None, ld, None, None, 0.0, M, 2 * M, None, 0, None)
    assert rc == gq.GQ_ELAUNCH, rc          # accepted, and there is nothing to launch on
"""


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("name,group", [("gq_act_wgrad", 0), ("gq_act_wgrad", 128),
                                        ("gq_block_wgrad", 128)])
def test_any_stride_without_rows(name, group, dtype):
    # the gradients are no real addresses: no GPU may be there to write to them
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="",
               CUDA_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", CALL.format(name=name, group=group, dtype=dtype)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


def test_room_of_no_rows_under_ubsan(tmp_path):
    """The rule itself, with division by zero and overflow checked."""
    src, exe = tmp_path / "room.cpp", str(tmp_path / "room")
    src.write_text('#include <initializer_list>\n#include "act_bounds.hpp"\n'
                   "int main(int argc, char**) {\n"
                   "  const int64_t none = argc - 1;\n"
                   "  for (int64_t ld : {none, none - 5, none + 1, (int64_t)1 << 39})\n"
                   "    if (gq::rows_with_room(none, ld, 7) != 0) return 1;\n"
                   "  return gq::rows_with_room(20 + none, 3, 7) == 17 ? 0 : 2;\n"
                   "}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "communication_efficient_gradient_amd", "csrc"),
                    str(src), "-o", exe], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0
