"""What the launches of linear and gated layers are passed (CPU checks, no GPU): every product's blocks cover its outputs and its
whole sum, once; every matrix that a call leaves in its workspace lies inside the size that was asked for, apart from those that
are still read; forward and backward calls, from one token to as many as the header allows."""
import ctypes
import json
import os
import random
import re
import shutil
import subprocess
import sys

import pytest

import mxfp4_precision_numerics_amd as mxq
import test_dense_launches as sizes
from test_dense_launches import MOST, gated, gated_back, linear, linear_back

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WS = 1 << 44  # the workspace's stand-in address: far from every other one
Z, DX, DW = 7, 14, 16  # places of a backward call's arguments
i32, i64, u32, u64, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_uint64
PRODUCT = [("A", p), ("B", p), ("lda", i64), ("ldb", i64), ("M", i64), ("N", i64), ("K", i64), ("m_from", i64), ("n_from", i64),
           ("ntm", i64), ("ntn", i64), ("first", u32), ("splits", i32), ("per", i64), ("pairs", i64), ("stride", i64),
           ("act", i32), ("bias", p), ("residual", p), ("ldr", i64), ("out", p), ("ldo", i64), ("f32", i32), ("nt", i32), ("z", p),
           ("ldz", i64), ("dh", p), ("ldh", i64), ("part", p)]
SUMS = [("p", p), ("ld", i64), ("rows", i64), ("N", i64), ("f32", i32), ("add", i32), ("out", p)]
BACK = [("dy", p), ("z", p), ("dz", p), ("ld_dy", i64), ("ld_z", i64), ("ld_dz", i64), ("T", i64), ("N", i64), ("rows", i64),
        ("part", p), ("act", i32)]
COUNT = [("n", u32)]
# a kernel's arguments; the first that its name holds
KERNELS = {"k_linear_grads_pipe": [PRODUCT, PRODUCT, SUMS, COUNT, COUNT, COUNT], "k_linear_grads": [PRODUCT, PRODUCT, SUMS, COUNT, COUNT, COUNT],
           "k_linear_join_two": [PRODUCT, PRODUCT, COUNT], "k_linear_join": [PRODUCT], "k_linear_rows": [PRODUCT],
           "k_linear_gemm": [PRODUCT], "k_linear_pipe": [PRODUCT], "k_linear_stream": [PRODUCT], "k_act_back": [BACK],
           "k_column_sums": [SUMS], "k_zero_rows": []}
CHILD = """
import ctypes, json, sys
R = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
class Record(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 160), ("grid", ctypes.c_uint32 * 3), ("block", ctypes.c_uint32 * 3),
                ("lds", ctypes.c_uint64), ("launch", ctypes.c_int32)]
R.record.restype = ctypes.POINTER(Record)
R.argument.restype = ctypes.POINTER(ctypes.c_ubyte)
kinds, calls = json.load(sys.stdin)
for part, lengths in kinds:
    R.expect(part.encode(), len(lengths), (ctypes.c_int * max(1, len(lengths)))(*lengths))
from mxfp4_precision_numerics_amd import dense
L = dense._lib()
out = []
for name, args in calls:
    R.forget()
    status = getattr(L, name)(*args)
    seen = []
    for r in range(R.recorded()):
        c = R.record(r).contents
        lengths = next((n for part, n in kinds if part in c.name.decode()), [])
        seen.append([c.name.decode(), list(c.grid), list(c.block), [bytes(R.argument(r, i)[:n]).hex() for i, n in enumerate(lengths)]])
    out.append([status, seen])
json.dump(out, sys.stdout)
"""


def struct(fields):
    return type("S", (ctypes.Structure,), {"_fields_": fields})


def with_workspace(call):
    """The call on a workspace of the size that the library gives, at WS; and its sizes."""
    name, args = call
    back, paired = "backward" in name, "gated" in name
    at = 11 if back else 5 if paired else 8
    T, H, N = args[at:at + 3]
    size = getattr(sizes.dense._lib(), ("mxq_gated_linear" if paired else "mxq_linear") + "_workspace")(T, H, N, int(back))
    return (name, args[:-3] + [WS, size, None]), (T, H, N, size)


def drawn(n):
    rng = random.Random(7)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    out = []
    for k in range(n):
        T, H, N = log(1, 1 << 14), 8 * log(1, 1 << 12), 8 * log(1, 1 << 12)
        act = k % 5
        backward = [linear_back(T, H, N, act, [sizes.P, None][k % 2], k % 3 // 2), gated_back(T, H, N, [sizes.P, None][k % 2])]
        out += [linear(T, H, N, act, k % 2), gated(T, H, N)] + backward
        alone = DX if k % 3 else DW
        out += [(name, [None if i == alone else v for i, v in enumerate(args)]) for name, args in backward]
    return out


LISTED = [c for c in sizes.CASES if c[0].startswith(("mxq_linear", "mxq_gated")) and 0 not in c[1][5:13]] + [
    linear_back(16, 32768, 1424), linear_back(128, 4104, 11280), linear_back(512, 4096, 4096), linear_back(8192, 14336, 4096),
    linear_back(4096, 4096, 14336, 4), gated_back(8192, 4096, 14336), gated_back(300, 1 << 14, 1 << 14, None), linear(70, 4096, 8192),
    linear(16, 1 << 20, 64), linear(3770, 4112, 368), linear(8192, 7168, 256), gated(24, 4096, 2048), linear(MOST, 72, 264)]


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    lib = str(tmp_path_factory.mktemp("recorder") / "libarguments.so")
    r = subprocess.run([gcc, "-shared", "-fPIC", "-O1", "-Wall", os.path.join(ROOT, "tests", "launches", "arguments.c"), "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return lib


def seen(recorder, calls):
    kinds = [(part, [ctypes.sizeof(struct(f)) for f in fields]) for part, fields in KERNELS.items()]
    r = subprocess.run([sys.executable, "-c", CHILD, recorder], cwd=ROOT, input=json.dumps([kinds, calls]), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    for status, records in json.loads(r.stdout):
        assert status == 0
        yield [(name, grid, block, [struct(f).from_buffer_copy(bytes.fromhex(b)) for f, b in
                                    zip(next(v for k, v in KERNELS.items() if k in name), args)]) for name, grid, block, args in records]


def tile(name, w=False):
    """Rows and columns of the kernel's tile; of both gradients' kernels the first product's, `w`: the second's."""
    m = re.search(r"k_linear_pipeILi(\d+)E", name)
    if m:
        return int(m[1]), 256
    m = re.search(r"k_linear_grads_pipeILi(\d+)ELi(\d+)E", name)
    if m:
        return int(m[1 + w]), 256
    m = re.search(r"k_linear_stream(?:I|IN\w*?)\w*?(Wide|Quick)(\d+)E", name)
    if m:
        return (128 if m[1] == "Wide" else 32), int(m[2])
    if "k_linear_grads" in name:
        m = re.search(r"k_linear_gradsI(.*)EvNS", name)
        parts = re.findall(r"NS_\d*(Mid|Tiny)E|S\d*_", m[1])
        names = [x or None for x in parts]
        kind = names[w] if len(names) > 1 and names[w] else names[0]
        return (128, 128) if kind == "Mid" else (64, 64)
    for kind, n in (("3Mid", 128), ("4Tiny", 64), ("4Deep", 64), ("4Lone", 128)):
        if kind in name:
            return n, n
    raise AssertionError(name)


def ceil(a, b):
    return -(-a // b)


class Region:
    """Bytes of the workspace that hold a matrix."""

    def __init__(self, at, size):
        self.a, self.b = at - WS, at - WS + size

    def apart(self, other):
        return self.b <= other.a or other.b <= self.a


def part(g):
    return Region(g.part, g.splits * g.N * g.M * 4) if g.part and g.splits > 1 else None


def matrix(at, ld, rows, bytes_):
    return Region(at, (rows - 1) * ld + bytes_) if WS <= at < WS << 1 else None


def check_product(g, bm, bn, blocks):
    """blocks: (first, count) of the launches.  The part of the output that they write: m from, m to, n from, n to."""
    step = g.stride or bm
    assert step <= bm and g.ntm * step >= g.M - g.m_from > (g.ntm - 1) * step
    assert g.ntn * bn >= g.N - g.n_from > (g.ntn - 1) * bn
    assert g.splits >= 1 and g.per * g.splits * 64 >= g.K
    assert g.splits == 1 or g.part
    at = 0
    for first, count in blocks:
        assert first == at
        at += count
    assert at == g.ntm * g.ntn * g.splits
    return g.m_from, g.M, g.n_from, g.N


def check_call(paired, info, records):
    T, H, N, size = info
    rows_of_w = 2 * N if paired else N
    products = []  # (kind, K, the part of its output that a launch writes)
    k = 0
    while k < len(records):
        name, grid, block, args = records[k]
        k += 1
        if "k_act_back" in name:
            b = args[0]
            assert grid[0] * 512 >= b.N and b.rows % 8 == 0 and grid[1] * b.rows >= b.T > (grid[1] - 1) * b.rows
            dz = matrix(b.dz, b.ld_dz, b.T, rows_of_w * 2) if b.dz else None
            sums = Region(b.part, grid[1] * b.N * 4) if b.part else None
            together = [r for r in (dz, sums) if r]
        elif "k_column_sums" in name:
            b = args[0]
            assert grid[0] * 32 >= b.N
            together = [matrix(b.p, b.ld, b.rows, b.N * (4 if b.f32 else 2))]
        elif "k_linear_rows" in name:
            assert T <= 4 and grid[0] * 8 >= N
            products.append(("forward", H, (0, rows_of_w, 0, T)))
            together = [matrix(args[0].out, args[0].ldo, T, rows_of_w * 2)]
        elif "k_linear_join_two" in name:
            x, w, nx = args[0], args[1], args[2].n
            for q, blocks in ((x, nx), (w, grid[0] - nx)):
                assert blocks == (ceil(q.N * (q.M // 8), 256) if q.splits > 1 else 0)
            together = [part(x), part(w)]
        elif "k_linear_join" in name:
            q, chunks = args[0], args[0].N * ((args[0].pairs or args[0].M) // 8)
            total = grid[0]
            while k < len(records) and "k_linear_join" in records[k][0] and records[k][3][0].first == total:
                total += records[k][1][0]
                k += 1
            assert total * 256 >= chunks and q.splits > 1
            together = [part(q), matrix(q.out, q.ldo, q.N, q.M * 2)]
        elif "k_linear_grads" in name:
            x, w, b = args[:3]
            sums = ceil(b.N, 32) if b.out else 0
            nx, nw = (q.ntm * q.ntn * q.splits for q in (x, w))
            assert grid[0] == sums + nx + nw
            assert args[3 if "pipe" in name else 4].n == (nw if args[5].n else nx)  # of the first product
            assert args[4].n == nx + nw if "pipe" in name else args[3].n == sums
            for q, second in ((x, False), (w, True)):
                at = check_product(q, *tile(name, second), [(0, q.ntm * q.ntn * q.splits)])
                products.append(("dw" if second else "dx", q.K, at))
            together = [part(x), part(w), matrix(x.B, x.ldb, x.N, x.K * 2)]
            assert x.B == w.B and x.ldb == w.ldb
            if b.out:
                together.append(matrix(b.p, b.ld, b.rows, b.N * (4 if b.f32 else 2)) if b.p != x.B else None)
        else:
            q = args[0]
            blocks = [(q.first, grid[0])]
            while k < len(records) and records[k][0] == name and records[k][3][0].first:  # the rest of a launch too large for one
                blocks.append((records[k][3][0].first, records[k][1][0]))
                k += 1
            at = check_product(q, *tile(name), blocks)
            flags = re.findall(r"Lb([01])E", name)  # A, B transposed, paired; a streaming kernel's: A, paired
            kind = "forward" if flags[0] == "0" else "dw" if "stream" not in name and flags[1] == "1" else "dx"
            products.append((kind, q.K, at))
            together = [part(q), matrix(q.B, q.ldb, q.N if kind != "dw" else q.K, (q.K if kind != "dw" else q.N) * 2),
                        matrix(q.out, q.ldo, q.N, q.M * 2)]
        together = [r for r in together if r]
        for i, a in enumerate(together):
            assert 0 <= a.a and a.b <= size, (name, a.a, a.b, size)
            assert all(a.apart(b) for b in together[:i]), name
    return products


def covered(parts):
    """The size that rectangles make up, if they do so without overlaps."""
    M, N = max(m for _, m, _, _ in parts), max(n for _, _, _, n in parts)
    for i, (a, b, c, d) in enumerate(parts):
        assert all(b <= e or f <= a or d <= g or h <= c for e, f, g, h in parts[:i])
    assert sum((b - a) * (d - c) for a, b, c, d in parts) == M * N
    return M, N


def check(recorder, calls):
    pairs = [with_workspace(c) for c in calls]
    for ((name, args), info), records in zip(pairs, seen(recorder, [c for c, _ in pairs])):
        T, H, N, _ = info
        back, paired = "backward" in name, "gated" in name
        rows = 2 * N if paired else N
        products = check_call(paired, info, records)
        wanted = {}
        if not back or paired and args[Z] is None:
            wanted["forward"] = (rows, T, H)
        if back and args[DX] is not None:
            wanted["dx"] = (H, T, rows)
        if back and args[DW] is not None:
            wanted["dw"] = (H, rows, T)
        assert {kind for kind, _, _ in products} == set(wanted), (name, info, products)
        for kind, (M, n, K) in wanted.items():
            mine = [at for k, length, at in products if k == kind and length == K]
            assert covered(mine) == (M, n), (name, info, kind, mine)


def test_listed_calls(recorder):
    check(recorder, LISTED)


def test_drawn_calls(recorder):
    check(recorder, drawn(250))
