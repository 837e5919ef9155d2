"""The host code of the 8-bit floating point products and the optimizer (csrc/step_api.hip) built with
the address and undefined-behaviour sanitizers for the host side only, running
the refusal tests (tests/test_step_abi.py, which reach no kernel launch) in a
child process."""
import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_step_host_code_under_asan_ubsan():
    from communication_efficient_gradient_amd import build as lib_build
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    hipcc = shutil.which("hipcc") or os.path.join(rocm, "bin", "hipcc")
    clang = os.path.join(rocm, "llvm", "bin", "clang++")
    out = os.path.join(ROOT, "_build", "sanitize")
    os.makedirs(out, exist_ok=True)
    objdir = os.path.join(ROOT, "_build", "libgq")
    others = [s[:-4] for s in lib_build.SOURCES if s != "step_api.hip"]
    if not all(os.path.exists(os.path.join(objdir, o + ".o")) for o in others):
        lib_build.build()
    host = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined",
                 "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"):
        host += ["-Xarch_host", flag]
    obj, lib = os.path.join(out, "step_api_asan.o"), os.path.join(out, "libgq_step_asan.so")
    flags = [f for f in lib_build.HIPFLAGS if f != "-O3"]
    subprocess.run([hipcc, *flags, "-O1", "-g", *host, "-c",
                    os.path.join(lib_build.CSRC, "step_api.hip"), "-o", obj],
                   check=True, capture_output=True)
    subprocess.run([clang, "-shared", "-fPIC", "-fsanitize=address,undefined",
                    "-shared-libsan", obj,
                    *[os.path.join(objdir, o + ".o") for o in others],
                    f"-L{rocm}/lib", "-lamdhip64", f"-Wl,-rpath,{rocm}/lib", "-o", lib],
                   check=True, capture_output=True)
    rt = subprocess.run([clang, "-print-file-name=libclang_rt.asan-x86_64.so"],
                        capture_output=True, text=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0", GQ_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p",
                        "no:cacheprovider", "-m", "not gpu",
                        os.path.join("tests", "test_step_abi.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert " passed" in r.stdout
