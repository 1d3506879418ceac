"""The host validation of include/mxq_dense.h built with AddressSanitizer and
UndefinedBehaviorSanitizer, its tests run against that build in a child
process."""
import glob
import os
import shutil
import subprocess

import pytest

from test_sanitized import ROOT, _run_child


def test_dense_validation_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    rt = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not os.path.exists(hipcc) or not rt:
        pytest.skip("hipcc or clang's AddressSanitizer runtime is not installed")
    lib = str(tmp_path / "libmxq_dense_san.so")
    csrc = os.path.join(ROOT, "mxfp4_precision_numerics_amd", "csrc")
    stubs = os.path.join(ROOT, "tests", "sanitize")
    sources = [os.path.join(csrc, f) for f in ("mxq_api.hip", "train_api.hip", "dense_api.hip")]
    sources += [os.path.join(stubs, f) for f in ("abi_stubs.hip", "train_stubs.hip", "dense_stubs.hip")]
    # host code only is instrumented (each -fsanitize after -Xarch_host)
    cmd = [hipcc, "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-shared", "-O1", "-g",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           "-I", os.path.join(ROOT, "include"), *sources, "-o", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    code = ("import sys, pytest\n"
            "import mxfp4_precision_numerics_amd as m\n"
            f"m.LIB_PATH = {lib!r}\n"
            "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', 'tests/test_dense_checks.py']))\n")
    out = _run_child(code, {"LD_PRELOAD": rt[-1]})
    assert " passed" in out
