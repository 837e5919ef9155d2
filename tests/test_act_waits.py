"""The weight gradient's kernels leave the wait for their copies to LDS to the
compiler, which has to place it before each barrier that hands the copies over.
This reads the assembly of a build and follows the memory operations in flight
up to every barrier (no GPU needed)."""
import os
import re
import subprocess

import pytest


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from communication_efficient_gradient_amd import build as lib_build
    out = str(tmp_path_factory.mktemp("waits") / "act_wgrad.s")
    subprocess.run([lib_build.hipcc(), *lib_build.HIPFLAGS, "--cuda-device-only", "-S",
                    os.path.join(lib_build.CSRC, "act_wgrad.hip"), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    # k_act_wgrad<T, COPY = true, ...>
    found = {}
    for part in re.split(r"\n(?=_ZN\S+:)", text):
        name = part.split(":", 1)[0]
        if re.search(r"11k_act_wgradI\w*?Lb1E", name):
            found[name] = [line.strip() for line in part.splitlines()]
    return found


def unwaited(lines):
    """Barriers that a copy to LDS may still be in flight at, and the number of
    barriers that copies were in flight before."""
    flight, bad, handed, copies = [], 0, 0, 0
    for line in lines:
        if re.match(r"(buffer|global|flat)_(load|store|atomic)", line):
            copy = line.startswith("buffer_load") and line.split(";")[0].rstrip().endswith("lds")
            flight.append(copy)
            copies += copy
        elif line.startswith("s_waitcnt"):
            m = re.search(r"vmcnt\((\d+)\)", line)
            if m and len(flight) > int(m[1]):       # in the order of issue
                flight = flight[len(flight) - int(m[1]):]
        elif line.startswith("s_barrier"):
            bad += any(flight)
            handed += copies > 0
            copies = 0
    return bad, handed


def test_copies_have_arrived_at_every_barrier(kernels):
    assert len(kernels) == 4                        # bf16 and fp16, two tiles
    for name, lines in kernels.items():
        bad, handed = unwaited(lines)
        # before the first step, twice in the loop over pairs of steps, last step
        assert handed >= 4, name
        assert bad == 0, name


def test_a_missing_wait_is_seen(kernels):
    for lines in kernels.values():
        waits = [i for i, line in enumerate(lines) if "vmcnt" in line]
        assert any(unwaited(lines[:i] + lines[i + 1:])[0] for i in waits)
