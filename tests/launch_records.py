"""What the training-step calls launch, noted by a stand-in for the HIP runtime
(tests/launches/recorder.c) in a child process: no GPU is involved."""
import json
import os
import shutil
import subprocess
import sys

import pytest

import mxfp4_precision_numerics_amd as mxq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import ctypes, json, sys
class Record(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 160), ("grid", ctypes.c_uint32 * 3), ("block", ctypes.c_uint32 * 3),
                ("lds", ctypes.c_uint64), ("launch", ctypes.c_int32)]
R = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
R.record.restype = ctypes.POINTER(Record)
from mxfp4_precision_numerics_amd import training
assert "torch" not in sys.modules
L = training._lib()
out = []
for name, args in json.load(sys.stdin):
    R.forget()
    status = getattr(L, name)(*args)
    seen = [R.record(i).contents for i in range(R.recorded())]
    out.append([status, [dict(name=r.name.decode(), grid=list(r.grid), block=list(r.block), lds=r.lds, launch=r.launch)
                         for r in seen]])
json.dump(out, sys.stdout)
"""


def launches(tmp_path, calls):
    """[(status, records)] of calls (C function, arguments); addresses are never read."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    if not os.path.exists(mxq.LIB_PATH):
        from mxfp4_precision_numerics_amd import build
        build.build()
    lib = str(tmp_path / "librecorder.so")
    r = subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-Wall", os.path.join(ROOT, "tests", "launches", "recorder.c"),
                        "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([sys.executable, "-c", CHILD, lib], cwd=ROOT, input=json.dumps(calls), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    return json.loads(r.stdout)
