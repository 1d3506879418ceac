"""The training-step operators on the host: every function that
include/mxq_train.h declares is exported and bound with its parameters, the C
entry points refuse invalid arguments before any HIP call, and the binding
refuses a wrong tensor before the library is reached (CPU checks)."""
import ast
import os
import re

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from mxfp4_precision_numerics_amd import training

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxq_train.h")
OK, ENULL, ESHAPE, EALIGN, EFMT = 0, -1, -2, -3, -4
P = 0x10000  # a 16-byte aligned stand-in address: never dereferenced here
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mxq.LIB_PATH):
        from mxfp4_precision_numerics_amd import build
        build.build()
    return training._lib()


def declared():
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(mxq_\w+)\s*\(", text, re.M)))


def test_every_declared_function_is_exported_and_bound(L):
    text = open(HEADER).read()
    names = declared()
    assert len(names) == 11
    for name in names:
        m = re.search(r"^(?:int|int64_t) " + name + r"\s*\(([^;]*)\);", text, re.S | re.M)
        params = [p for p in m.group(1).split(",") if p.strip()]
        assert len(getattr(L, name).argtypes) == len(params), name


def test_constants_match_the_header():
    text = open(HEADER).read()
    assert f"MXQ_CLIP_CHUNK = {mxq.GradientSet.CHUNK}" in text
    assert f"MXQ_CLIP_PARTS = {mxq.GradientSet.PARTS}" in text


def test_topk_validation(L):
    f = lambda z=P, src=0, T=4, E=16, ld=16, k=2, ids=P, w=P: L.mxq_moe_topk(z, src, T, E, ld, k, 0, ids, w, None)
    assert f(src=2) == EFMT
    assert f(T=-1) == f(E=0, ld=0) == f(E=1025, ld=1025) == f(k=0) == f(k=17) == f(ld=15) == ESHAPE
    assert f(E=100, ld=100, k=65) == ESHAPE
    assert f(z=None) == f(ids=None) == f(w=None) == ENULL
    assert f(z=P + 2) == f(ids=P + 2) == f(w=P + 1) == EALIGN
    assert f(T=0) == f(T=0, z=None, ids=None, w=None) == OK
    b = lambda z=P, T=4, ld=16, ld_d=16, ids=P, dw=P, dz=P: L.mxq_moe_topk_backward(z, 1, T, 16, ld, ids, 2, 1, dw, dz,
                                                                                     ld_d, None)
    assert b(ld=8) == b(ld_d=15) == ESHAPE
    assert b(z=None) == b(ids=None) == b(dw=None) == b(dz=None) == ENULL
    assert b(z=P + 1) == b(dz=P + 1) == b(dw=P + 2) == EALIGN
    assert b(T=0, z=None, ids=None, dw=None, dz=None) == OK


def test_sort_validation(L):
    ws = L.mxq_moe_sort_workspace
    assert ws(-1, 1, 1) == ws(1, 0, 1) == ws(1, 1, 0) == ws(1, 1, 4097) == ws(1 << 30, 2, 1) == ESHAPE
    assert ws(BIG, BIG, 1) == ESHAPE
    assert ws(16, 8, 256) == 0 and ws(8192, 8, 256) > 0
    f = lambda ids=P, T=8192, k=8, G=256, off=P, src=P, pos=P, w=P, n=1 << 20: L.mxq_moe_sort(ids, T, k, G, off, src, pos,
                                                                                          w, n, None)
    assert f(ids=None) == f(off=None) == f(pos=None) == f(w=None) == ENULL
    assert f(n=100) == f(G=0) == f(T=-1) == ESHAPE
    assert f(off=P + 4) == f(ids=P + 1) == f(src=P + 2) == f(pos=P + 2) == f(w=P + 8) == EALIGN


def test_dispatch_validation(L):
    f = lambda x=P, src=1, T=4, C=64, ld=64, pos=P, k=2, fmt=0, R=8, q=P, s=P: L.mxq_moe_dispatch_mx(
        x, src, T, C, ld, pos, k, fmt, R, q, s, None)
    assert f(fmt=3) == f(src=5) == EFMT
    assert f(C=48, ld=48) == f(ld=32) == f(T=-1) == f(R=-1) == f(k=0) == f(T=1 << 30, C=1024, ld=1024) == ESHAPE
    assert f(x=None) == f(pos=None) == f(q=None) == f(s=None) == ENULL
    assert f(x=P + 8) == f(ld=68) == f(q=P + 4) == f(pos=P + 2) == EALIGN
    assert f(T=0, x=None, pos=None) == f(R=0, q=None, s=None) == f(C=0, ld=0) == OK


def test_combine_validation(L):
    f = lambda x=P, src=1, R=8, C=64, ld=64, pos=P, T=4, k=2, w=P, y=P, ldy=64: L.mxq_moe_combine(
        x, src, R, C, ld, pos, T, k, w, y, ldy, None)
    assert f(src=2) == EFMT
    assert f(C=60, ld=60, ldy=60) == f(ld=32) == f(ldy=32) == f(T=-1) == f(k=0) == f(T=1 << 30) == ESHAPE
    assert f(x=None) == f(pos=None) == f(y=None) == ENULL
    assert f(x=P + 8) == f(y=P + 8) == f(ld=68) == f(ldy=68) == f(w=P + 2) == EALIGN
    assert f(T=0, pos=None, y=None) == OK
    b = lambda dy=P, T=4, C=64, ld=64, pos=P, k=2, w=P, x=P, ldx=64, R=8, dx=P, ldd=64, dw=P: (
        L.mxq_moe_combine_backward(dy, 1, T, C, ld, pos, k, w, x, ldx, R, dx, ldd, dw, None))
    assert b(k=65) == b(ld=32) == b(ldx=32) == b(ldd=32) == b(C=60) == ESHAPE
    assert b(dx=None, dw=None) == b(x=None) == b(pos=None) == b(dy=None) == ENULL
    assert b(dy=P + 4) == b(x=P + 8) == b(dx=P + 8) == b(ldd=68) == b(dw=P + 1) == EALIGN
    assert b(T=0, dy=None, pos=None) == OK


def test_cross_entropy_validation(L):
    ws = L.mxq_linear_cross_entropy_workspace
    assert ws(4, 12, 100, 0) == ws(4, 0, 100, 0) == ws(-1, 64, 100, 0) == ws(4, 64, 0, 0) == ESHAPE
    assert ws(1 << 31, 64, 100, 0) == ws(4, 64, 1 << 31, 1) == ESHAPE
    assert 0 < ws(300, 64, 1000, 0) <= ws(300, 64, 1000, 1)
    f = lambda x=P, ldx=64, w=P, ldw=64, t=P, T=4, H=64, V=100, lo=P, ls=P, s=P, n=BIG: L.mxq_linear_cross_entropy(
        x, ldx, w, ldw, t, T, H, V, lo, ls, s, n, None)
    assert f(x=None) == f(w=None) == f(t=None) == f(lo=None) == f(ls=None) == f(s=None) == ENULL
    assert f(ldx=56) == f(ldw=56) == f(n=16) == f(V=0) == f(ldx=1 << 22) == ESHAPE
    assert f(ldx=68) == f(x=P + 8) == f(w=P + 2) == f(s=P + 8) == f(t=P + 4) == f(lo=P + 2) == EALIGN
    assert f(T=0, x=None, t=None, lo=None, ls=None, s=None) == OK
    b = lambda x=P, T=4, ls=P, dl=P, dx=P, lddx=64, dw=P, lddw=64, s=P, n=BIG: L.mxq_linear_cross_entropy_backward(
        x, 64, P, 64, P, T, 64, 100, ls, dl, dx, lddx, dw, lddw, s, n, None)
    assert b(x=None) == b(ls=None) == b(dl=None) == b(s=None) == b(dx=None, dw=None) == ENULL
    assert b(lddx=56) == b(lddw=56) == b(n=16) == ESHAPE
    assert b(lddx=68) == b(dx=P + 8) == b(dw=P + 8) == b(ls=P + 2) == EALIGN
    assert b(T=0, dx=None, dw=None) == OK


def test_clip_validation(L):
    f = lambda t=P, n=2, c=P, ch=2, mx=1.0, norm=P, parts=P: L.mxq_clip_grad_norm(t, n, c, ch, mx, norm, parts, None)
    assert f(t=None) == f(c=None) == f(norm=None) == f(parts=None) == ENULL
    assert f(n=-1) == f(ch=-1) == f(mx=-1.0) == f(mx=float("nan")) == f(mx=float("inf")) == ESHAPE
    assert f(t=P + 4) == f(c=P + 2) == f(norm=P + 2) == f(parts=P + 4) == EALIGN


class _Sizes:
    """Answers the size functions and refuses every other call."""

    def __getattr__(self, name):
        class F:
            def __call__(self, *a):
                if name.endswith("_workspace"):
                    return 64
                raise AssertionError(f"{name} was reached with invalid arguments")
        return F()


@pytest.fixture
def stub(monkeypatch):
    monkeypatch.setattr(mxq, "_lib", _Sizes())
    monkeypatch.setattr(training, "_bound", mxq._lib)


BF = torch.bfloat16
z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)
i32 = lambda *s: z(*s, dtype=torch.int32)
i64 = lambda *s: z(*s, dtype=torch.int64)
bf = lambda *s: z(*s, dtype=BF)
u8 = lambda *s: z(*s, dtype=torch.uint8)
WS = u8(64)


def cases():
    """(label, call, expected exception) - each call has exactly one defect."""
    lce = mxq.linear_cross_entropy
    back = mxq.linear_cross_entropy_backward
    return [
        ("topk logits dtype", lambda: mxq.moe_topk(z(4, 16, dtype=torch.float16), i32(4, 2), z(4, 2)), TypeError),
        ("topk logits stride", lambda: mxq.moe_topk(z(16, 4).t(), i32(4, 2), z(4, 2)), ValueError),
        ("topk ids dtype", lambda: mxq.moe_topk(z(4, 16), i64(4, 2), z(4, 2)), TypeError),
        ("topk ids short", lambda: mxq.moe_topk(z(4, 16), i32(3, 2), z(4, 2)), ValueError),
        ("topk weights short", lambda: mxq.moe_topk(z(4, 16), i32(4, 2), z(4, 1)), ValueError),
        ("topk host", lambda: mxq.moe_topk(z(4, 16), i32(4, 2), z(4, 2)), ValueError),
        ("topk back type", lambda: mxq.moe_topk_backward(z(4, 16), i32(4, 2), z(4, 2), bf(4, 16)), TypeError),
        ("topk back narrow", lambda: mxq.moe_topk_backward(z(4, 16), i32(4, 2), z(4, 2), z(4, 15)), ValueError),
        ("sort off short", lambda: mxq.moe_sort(i32(4, 2), 8, i64(8), i32(8), i32(4, 2), WS), ValueError),
        ("sort off dtype", lambda: mxq.moe_sort(i32(4, 2), 8, i32(9), i32(8), i32(4, 2), WS), TypeError),
        ("sort pos short", lambda: mxq.moe_sort(i32(4, 2), 8, i64(9), i32(8), i32(3, 2), WS), ValueError),
        ("sort src short", lambda: mxq.moe_sort(i32(4, 2), 8, i64(9), i32(7), i32(4, 2), WS), ValueError),
        ("sort workspace", lambda: mxq.moe_sort(i32(4, 2), 8, i64(9), i32(8), i32(4, 2)), ValueError),
        ("sort workspace short", lambda: mxq.moe_sort(i32(4, 2), 8, i64(9), None, i32(4, 2), u8(63)), ValueError),
        ("dispatch q short", lambda: mxq.moe_dispatch_mx(bf(4, 64), i32(4, 2), 0, u8(8, 63), u8(8, 2)), ValueError),
        ("dispatch s short", lambda: mxq.moe_dispatch_mx(bf(4, 64), i32(4, 2), 0, u8(8, 64), u8(8, 1)), ValueError),
        ("dispatch pos tokens", lambda: mxq.moe_dispatch_mx(bf(4, 64), i32(2, 4), 0, u8(8, 64), u8(8, 2)), ValueError),
        ("dispatch pos dtype", lambda: mxq.moe_dispatch_mx(bf(4, 64), i64(4, 2), 0, u8(8, 64), u8(8, 2)), TypeError),
        ("dispatch host", lambda: mxq.moe_dispatch_mx(bf(4, 64), i32(4, 2), 0, u8(8, 64), u8(8, 2)), ValueError),
        ("combine y type", lambda: mxq.moe_combine(bf(8, 64), i32(4, 2), z(4, 64)), TypeError),
        ("combine y short", lambda: mxq.moe_combine(bf(8, 64), i32(4, 2), bf(3, 64)), ValueError),
        ("combine weights short", lambda: mxq.moe_combine(bf(8, 64), i32(4, 2), bf(4, 64), z(4, 1)), ValueError),
        ("combine back nothing", lambda: mxq.moe_combine_backward(bf(4, 64), i32(4, 2)), ValueError),
        ("combine back rows", lambda: mxq.moe_combine_backward(bf(4, 64), i32(4, 2), dweights=z(4, 2)), ValueError),
        ("combine back type", lambda: mxq.moe_combine_backward(bf(4, 64), i32(4, 2), z(8, 64)), TypeError),
        ("combine back narrow", lambda: mxq.moe_combine_backward(bf(4, 64), i32(4, 2), bf(8, 32)), ValueError),
        ("loss x dtype", lambda: lce(z(4, 64), bf(9, 64), i64(4), z(4), z(4), WS), TypeError),
        ("loss w width", lambda: lce(bf(4, 64), bf(9, 72), i64(4), z(4), z(4), WS), ValueError),
        ("loss targets dtype", lambda: lce(bf(4, 64), bf(9, 64), i32(4), z(4), z(4), WS), TypeError),
        ("loss targets short", lambda: lce(bf(4, 64), bf(9, 64), i64(3), z(4), z(4), WS), ValueError),
        ("loss lse short", lambda: lce(bf(4, 64), bf(9, 64), i64(4), z(4), z(3), WS), ValueError),
        ("loss workspace short", lambda: lce(bf(4, 64), bf(9, 64), i64(4), z(4), z(4), u8(8)), ValueError),
        ("loss host", lambda: lce(bf(4, 64), bf(9, 64), i64(4), z(4), z(4), WS), ValueError),
        ("loss back nothing", lambda: back(bf(4, 64), bf(9, 64), i64(4), z(4), z(4), None, None, WS), ValueError),
        ("loss back dx type", lambda: back(bf(4, 64), bf(9, 64), i64(4), z(4), z(4), z(4, 64), None, WS), TypeError),
        ("loss back dw short", lambda: back(bf(4, 64), bf(9, 64), i64(4), z(4), z(4), None, bf(8, 64), WS), ValueError),
        ("clip none", lambda: mxq.GradientSet([]), ValueError),
        ("clip dtype", lambda: mxq.GradientSet([z(4, dtype=torch.float16)]), TypeError),
        ("clip strided", lambda: mxq.GradientSet([z(4, 8).t()]), ValueError),
        ("clip out type", lambda: mxq.GradientSet([z(4)], [bf(4)]), TypeError),
        ("clip out short", lambda: mxq.GradientSet([z(4)], [z(3)]), ValueError),
        ("clip out count", lambda: mxq.GradientSet([z(4)], []), ValueError),
        ("clip host", lambda: mxq.GradientSet([z(4)]), ValueError),
    ]


@pytest.mark.parametrize("label,call,exc", cases(), ids=[c[0] for c in cases()])
def test_invalid_tensor_raises_before_the_library(stub, label, call, exc):
    with pytest.raises(exc) as e:
        call()
    assert ("GPU tensor" in str(e.value)) == ("host" in label), str(e.value)


def test_missing_library_raises(monkeypatch):
    monkeypatch.setattr(mxq, "LIB_PATH", os.path.join(ROOT, "does-not-exist", "libmxq.so"))
    monkeypatch.setattr(mxq, "_lib", None)
    for call in (lambda: mxq.moe_topk(z(4, 16), i32(4, 2), z(4, 2)),
                 lambda: mxq.linear_cross_entropy_workspace(4, 64, 100),
                 lambda: mxq.moe_combine(bf(8, 64), i32(4, 2), bf(4, 64))):
        with pytest.raises(RuntimeError, match="is missing"):
            call()


def test_public_names():
    tree = ast.parse(open(os.path.join(os.path.dirname(mxq.__file__), "training.py")).read())
    for node in tree.body:
        if isinstance(node, (ast.FunctionDef, ast.ClassDef)) and not node.name.startswith("_"):
            assert getattr(mxq, node.name) is getattr(training, node.name)
            assert ast.get_docstring(node), node.name
