"""The weight gradient from the 8-bit floating point form leaves the wait for its
copies to LDS to the compiler, as the one from 8-bit integers does; and the
products wait by themselves, so the compiler must not add waits of its own to
their loops (no GPU needed)."""
import os
import re
import subprocess

import pytest

from tests.test_act_waits import unwaited


def assembly(tmp_path_factory, name):
    from communication_efficient_gradient_amd import build as lib_build
    out = str(tmp_path_factory.mktemp("waits") / (name + ".s"))
    subprocess.run([lib_build.hipcc(), *lib_build.HIPFLAGS, "--cuda-device-only", "-S",
                    os.path.join(lib_build.CSRC, name + ".hip"), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    return {p.split(":", 1)[0]: [line.strip() for line in p.splitlines()]
            for p in re.split(r"\n(?=_ZN\S+:)", text)}


@pytest.fixture(scope="module")
def gradients(tmp_path_factory):
    """k_fp8_wgrad<T, COPY = true, ...>"""
    return {n: lines for n, lines in assembly(tmp_path_factory, "fp8_wgrad").items()
            if re.search(r"11k_fp8_wgradI\w*?Lb1E", n)}


def test_copies_have_arrived_at_every_barrier(gradients):
    assert len(gradients) == 4                      # bf16 and fp16, two tiles
    for name, lines in gradients.items():
        bad, handed = unwaited(lines)
        # before the first step, twice in the loop over pairs of steps, last step
        assert handed >= 4, name
        assert bad == 0, name


def test_a_missing_wait_is_seen(gradients):
    for lines in gradients.values():
        waits = [i for i, line in enumerate(lines) if "vmcnt" in line]
        assert any(unwaited(lines[:i] + lines[i + 1:])[0] for i in waits)


def test_products_wait_for_no_more_than_they_ask(tmp_path_factory):
    """Between the first and the last product of a tile, copies are only waited
    for in the inline assembly."""
    kernels = {n: lines for n, lines in assembly(tmp_path_factory, "fp8_linear").items()
               if re.search(r"12k_fp8_linearI", n)}
    assert len(kernels) == 12       # three types, three tiles, the smallest by two teams
    for name, lines in kernels.items():
        products = [i for i, line in enumerate(lines) if line.startswith("v_mfma")]
        inline = False
        for line in lines[products[0]:products[-1]]:
            if "ASMSTART" in line or "ASMEND" in line:
                inline = "ASMSTART" in line
            elif not inline and line.startswith("s_waitcnt"):
                assert "vmcnt" not in line, name
