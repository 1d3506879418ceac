"""Linear layers, gated layers and AdamW on the host: every function that include/mxq_dense.h declares is exported and
bound with its parameters, the C entry points refuse invalid arguments before any HIP call, and the binding refuses a
wrong tensor before the library is reached (CPU checks)."""
import os
import re

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from mxfp4_precision_numerics_amd import dense, training
from test_train_binding import on

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxq_dense.h")
OK, ENULL, ESHAPE, EALIGN, EFMT = 0, -1, -2, -3, -4
P = 0x10000  # a 16-byte aligned stand-in address: never dereferenced here
BIG, HUGE = 1 << 60, (1 << 63) - 1
BF, F32, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mxq.LIB_PATH):
        from mxfp4_precision_numerics_amd import build
        build.build()
    return dense._lib()


def test_every_declared_function_is_exported_and_bound(L):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(mxq_\w+)\s*\(", text, re.M)))
    assert len(names) == 8
    for name in names:
        m = re.search(r"^(?:int|int64_t) " + name + r"\s*\(([^;]*)\);", text, re.S | re.M)
        assert len(getattr(L, name).argtypes) == len([p for p in m.group(1).split(",") if p.strip()]), name


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name in ("NONE", "RELU", "SILU", "GELU", "GELU_TANH"):
        assert re.search(rf"MXQ_ACT_{name} = {getattr(mxq, 'ACT_' + name)}\b", text), name
    assert f"MXQ_STATE_BLOCK = {mxq.AdamW.BLOCK}" in text
    assert f"MXQ_CLIP_CHUNK = {mxq.AdamW.CHUNK}" in open(os.path.join(ROOT, "include", "mxq_train.h")).read()


def sizes_refused(f, width):
    most = 1 << 20 if width == "N" else 1 << 19
    for bad in (dict(T=-1), dict(T=(1 << 31) - 256), dict(H=0), dict(H=12), dict(H=(1 << 20) + 8), {width: 0}, {width: 20},
                {width: most + 8}, {width: -8}, dict(T=HUGE, H=HUGE), {width: HUGE}):
        assert f(**bad) == ESHAPE, bad


def test_workspace_sizes(L):
    for name, width in (("mxq_linear_workspace", "N"), ("mxq_gated_linear_workspace", "I")):
        f = lambda T=64, H=64, back=1, name=name, **k: getattr(L, name)(T, H, k.get(width, 64), back)
        sizes_refused(f, width)
        sizes_refused(lambda **k: f(back=0, **k), width)
        assert f(T=0) >= 0 and f(T=0, back=0) == 0
        assert f(T=(1 << 31) - 257, H=1 << 20, **{width: 1 << 19}) > 0


def test_linear_validation(L):
    def f(x=P, ldx=64, w=P, ldw=64, b=P, act=4, r=P, ldr=64, T=64, H=64, N=64, y=P, out=1, ldy=64, z=P, ldz=64, ws=P, n=BIG):
        return L.mxq_linear(x, ldx, w, ldw, b, act, r, ldr, T, H, N, y, out, ldy, z, ldz, ws, n, None)
    assert f(act=-1) == f(act=5) == f(out=2) == f(out=-1) == EFMT
    sizes_refused(f, "N")
    for bad in ("ldx", "ldw", "ldr", "ldy", "ldz"):
        assert f(**{bad: 56}) == f(**{bad: -64}) == f(**{bad: (2 << 20) + 8}) == f(**{bad: HUGE}) == ESHAPE, bad
        assert f(**{bad: 68}) == EALIGN, bad
    assert f(out=0, ldy=(1 << 20) + 8) == f(out=0, ldr=(1 << 20) + 8) == ESHAPE  # 4 MiB in floats
    assert f(x=None) == f(w=None) == f(y=None) == ENULL
    for bad in "xwryzb":
        assert f(**{bad: P + 8}) == EALIGN, bad
    need = L.mxq_linear_workspace(4, 16384, 64, 0)
    assert f(T=0) == f(T=0, x=None, w=None, y=None, ws=None) == OK
    split = dict(T=300, H=32768, ldx=32768, ldw=32768)  # a sum in parts
    assert L.mxq_linear_workspace(300, 32768, 64, 0) > 0 and need >= 0
    assert f(ws=None, **split) == ENULL and f(ws=P + 8, **split) == EALIGN
    assert f(n=L.mxq_linear_workspace(300, 32768, 64, 0) - 1, **split) == f(n=-1, **split) == ESHAPE


def test_linear_backward_validation(L):
    def f(x=P, ldx=64, w=P, ldw=64, dy=P, ldy=64, act=2, z=P, ldz=64, a=P, lda=64, T=64, H=64, N=64, dx=P, ldd=64, dw=P,
          out=1, ldg=64, db=P, acc=0, ws=P, n=BIG):
        return L.mxq_linear_backward(x, ldx, w, ldw, dy, ldy, act, z, ldz, a, lda, T, H, N, dx, ldd, dw, out, ldg, db, acc, ws,
                                     n, None)
    assert f(act=9) == f(out=2) == EFMT
    sizes_refused(f, "N")
    for bad in ("ldx", "ldw", "ldy", "ldz", "lda", "ldd", "ldg"):
        assert f(**{bad: 56}) == f(**{bad: (2 << 20) + 8}) == f(**{bad: HUGE}) == ESHAPE, bad
        assert f(**{bad: 68}) == EALIGN, bad
    assert f(dx=None, dw=None, db=None) == f(dx=None) == f(z=None) == f(x=None) == f(w=None) == f(dy=None) == ENULL
    assert f(dx=None, a=None, dw=None, db=None) == ENULL
    assert f(ws=None) == ENULL and f(n=0) == ESHAPE and f(ws=P + 8) == EALIGN
    for bad in ("x", "w", "dy", "z", "a", "dx", "dw", "db"):
        assert f(**{bad: P + 8}) == EALIGN, bad


def test_gated_validation(L):
    def f(x=P, ldx=64, w=P, ldw=64, act=2, T=64, H=64, I=64, h=P, ldh=64, z=P, ldz=128, ws=P, n=BIG):
        return L.mxq_gated_linear(x, ldx, w, ldw, act, T, H, I, h, ldh, z, ldz, ws, n, None)
    assert f(act=5) == EFMT
    sizes_refused(f, "I")
    for bad, at in (("ldx", 56), ("ldw", 56), ("ldh", 56), ("ldz", 120)):
        assert f(**{bad: at}) == f(**{bad: (2 << 20) + 8}) == f(**{bad: HUGE}) == ESHAPE, bad
        assert f(**{bad: at + 12}) == EALIGN, bad
    assert f(x=None) == f(w=None) == f(h=None) == ENULL
    assert f(x=P + 2) == f(w=P + 2) == f(h=P + 2) == f(z=P + 2) == EALIGN
    assert f(T=0, x=None, w=None, h=None) == OK

    def b(x=P, w=P, dh=P, ldh=64, act=2, z=P, ldz=128, a=P, lda=64, T=64, H=64, I=64, dx=P, ldd=64, dw=P, out=0, ldg=64, ws=P,
          n=BIG):
        return L.mxq_gated_linear_backward(x, 64, w, 64, dh, ldh, act, z, ldz, a, lda, T, H, I, dx, ldd, dw, out, ldg, 0, ws, n,
                                           None)
    assert b(act=-1) == b(out=3) == EFMT
    for bad, at in (("ldh", 56), ("ldz", 120), ("lda", 56), ("ldd", 56), ("ldg", 56)):
        assert b(**{bad: at}) == b(**{bad: HUGE}) == ESHAPE, bad
        assert b(**{bad: at + (10 if bad == "ldg" else 12)}) == EALIGN, bad
    assert b(dx=None, a=None, dw=None) == b(dx=None) == b(dh=None) == b(x=None) == b(w=None) == ENULL
    assert b(z=None, dw=None, x=None) == b(z=None, dx=None, a=None, w=None) == ENULL  # gate and up computed again
    assert b(ws=None) == ENULL and b(n=0) == ESHAPE


def test_adamw_validation(L):
    nan, inf = float("nan"), float("inf")

    def f(t=P, count=1, of=P, chunks=1, states=1, rate=0.1, rate_at=None, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1,
          step_at=None, norm=None, most=1.0):
        return L.mxq_adamw(t, count, of, chunks, states, rate, rate_at, b1, b2, eps, wd, step, step_at, norm, most, 0, None)
    assert f(states=2) == EFMT
    for bad in (dict(count=-1), dict(chunks=-1), dict(chunks=1 << 31), dict(count=1 << 31), dict(step=0), dict(step=-1)):
        assert f(**bad) == ESHAPE, bad
    for name in ("b1", "b2"):
        assert f(**{name: 1.0}) == f(**{name: -0.1}) == f(**{name: nan}) == ESHAPE
    assert f(eps=0.0) == f(eps=1e-39) == f(eps=nan) == f(eps=1e31) == f(eps=-1.0) == ESHAPE
    for name in ("wd", "most", "rate"):
        assert f(**{name: -1.0}) == f(**{name: nan}) == f(**{name: inf}) == ESHAPE, name
    assert f(t=None) == f(of=None) == ENULL
    assert f(t=P + 4) == f(of=P + 2) == f(rate_at=P + 2) == f(step_at=P + 4) == f(norm=P + 1) == EALIGN
    assert f(count=0, chunks=0, t=None, of=None) == OK
    # a rate and a number in memory take the place of these
    assert f(chunks=0, rate=nan, rate_at=P) == f(chunks=0, step=0, step_at=P) == OK


def test_grad_norm_validation(L):
    f = lambda t=P, count=1, of=P, chunks=1, norm=P, parts=P: L.mxq_grad_norm(t, count, of, chunks, norm, parts, None)
    assert f(count=-1) == f(chunks=-1) == f(chunks=1 << 31) == ESHAPE
    assert f(t=None) == f(of=None) == f(norm=None) == f(parts=None) == ENULL
    assert f(t=P + 4) == f(of=P + 2) == f(norm=P + 2) == f(parts=P + 4) == EALIGN


class _Reached(Exception):
    pass


class _Library:
    """Answers the size functions; any other call says that it was reached."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_workspace"):
                return 16
            raise _Reached(name)
        return call


@pytest.fixture
def stub(monkeypatch):
    """GPU 0 is the current one."""
    monkeypatch.setattr(mxq, "_lib", _Library())
    monkeypatch.setattr(training, "_bound", mxq._lib)
    monkeypatch.setattr(dense, "_bound", mxq._lib)
    monkeypatch.setattr(dense, "_sizes", {})
    monkeypatch.setattr(training, "_stream", lambda s, here: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


WS = ("workspace", (16,), U8)
CALLS = {
    "linear": [("x", (4, 16), BF), ("w", (24, 16), BF), ("y", (4, 24), F32), ("bias", (24,), F32), ("residual", (4, 24), F32),
               ("z", (4, 24), BF), WS],
    "linear_backward": [("x", (4, 16), BF), ("w", (24, 16), BF), ("dy", (4, 24), BF), ("dx", (4, 16), BF), ("dw", (24, 16), F32),
                        ("dbias", (24,), F32), ("z", (4, 24), BF), ("add", (4, 16), BF), WS],
    "gated_linear": [("x", (4, 16), BF), ("w", (48, 16), BF), ("h", (4, 24), BF), ("z", (4, 48), BF), WS],
    "gated_linear_backward": [("x", (4, 16), BF), ("w", (48, 16), BF), ("dh", (4, 24), BF), ("dx", (4, 16), BF),
                              ("dw", (48, 16), BF), ("z", (4, 48), BF), ("add", (4, 16), BF), WS],
}
NEEDED = {"linear": ("y", "workspace"), "linear_backward": ("dy", "workspace"), "gated_linear": ("h", "workspace"),
          "gated_linear_backward": ("dh", "workspace")}


def given(name, **other):
    return {**{n: on(0, *s, dtype=d) for n, s, d in CALLS[name]}, **other}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(stub, name):
    call = lambda where: getattr(mxq, name)(**{n: on(where(n), *s, dtype=d) for n, s, d in CALLS[name]})
    with pytest.raises(_Reached):
        call(lambda n: 0)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        call(lambda n: 1)
    for odd, _, _ in CALLS[name]:
        with pytest.raises(ValueError, match=f"^{odd} is on cuda:1"):
            call(lambda n: int(n == odd))
    with pytest.raises((ValueError, TypeError)):  # host tensors
        getattr(mxq, name)(**{n: torch.zeros(s, dtype=d) for n, s, d in CALLS[name]})


@pytest.mark.parametrize("name", CALLS)
def test_types_layouts_and_extents_are_refused(stub, name):
    f = getattr(mxq, name)
    for n, shape, dtype in CALLS[name]:
        if n != "workspace":  # bytes, whatever their type
            with pytest.raises(TypeError, match=n):
                f(**given(name, **{n: on(0, *shape, dtype=torch.float16)}))
        if len(shape) == 2:
            with pytest.raises(ValueError, match=n):  # columns not next to each other
                f(**given(name, **{n: on(0, *shape[::-1], dtype=dtype).t()}))
            for bad in ((shape[0], shape[1] + 8), (shape[0], shape[1] - 8), (shape[0] * shape[1],)):
                with pytest.raises(ValueError):
                    f(**given(name, **{n: on(0, *bad, dtype=dtype)}))
        if n not in ("x", "w"):  # these give the call its sizes
            with pytest.raises(ValueError, match=n):
                f(**given(name, **{n: on(0, shape[0] - 1, *shape[1:], dtype=dtype)}))
    for n in NEEDED[name]:
        with pytest.raises(ValueError, match=n):
            f(**given(name, **{n: None}))


def test_what_belongs_together(stub):
    with pytest.raises(TypeError, match="residual"):
        mxq.linear(**given("linear", residual=on(0, 4, 24, dtype=BF)))
    for name in ("linear_backward", "gated_linear_backward"):
        f, none = getattr(mxq, name), dict(dx=None, dw=None, add=None)
        if name == "linear_backward":
            none["dbias"] = None
        with pytest.raises(ValueError, match="required"):
            f(**given(name, **none))
        with pytest.raises(ValueError, match="dx is required"):
            f(**given(name, dx=None))
    with pytest.raises(ValueError, match="z is required"):
        mxq.linear_backward(**given("linear_backward", z=None), activation=mxq.ACT_GELU)
    with pytest.raises(_Reached):
        mxq.linear_backward(**given("linear_backward", z=None))
    with pytest.raises(_Reached):
        mxq.gated_linear_backward(**given("gated_linear_backward", z=None))
    with pytest.raises(ValueError, match="rows"):
        mxq.gated_linear(on(0, 4, 16, dtype=BF), on(0, 25, 16, dtype=BF), on(0, 4, 12, dtype=BF))


def test_views_with_a_row_pitch_are_taken(stub):
    wide = lambda r, c, dtype: torch.Tensor.as_subclass(on(0, r + 3, c + 32, dtype=dtype)[1:r + 1, 8:c + 8], type(on(0, 1)))
    for name in CALLS:
        t = {n: wide(*s, d) if len(s) == 2 else on(0, *s, dtype=d) for n, s, d in CALLS[name]}
        with pytest.raises(_Reached):
            getattr(mxq, name)(**t)


def lists(sizes=(40, 300), eight=True, p=F32, copies=True):
    make = lambda d: [on(0, n, dtype=d) for n in sizes]
    r = dict(params=make(p), grads=make(BF), m=make(U8 if eight else F32), v=make(U8 if eight else F32))
    if eight:
        r.update(m_scale=[on(0, -(-n // 128)) for n in sizes], v_scale=[on(0, -(-n // 128)) for n in sizes])
    if copies and p is F32:
        r["copies"] = [on(0, sizes[0], dtype=BF), None]
    return r


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
def test_an_update_set_refuses_what_does_not_fit(stub, eight):
    mxq.AdamW(**lists(eight=eight)), mxq.AdamW(**lists(eight=eight, p=BF))
    for name in lists(eight=eight):
        for bad, error in ((on(0, 41), (TypeError, ValueError)), (on(0, 40, dtype=torch.float16), TypeError),
                           (None, ValueError)):
            a = lists(eight=eight)
            if name == "copies" and bad is None:
                continue
            a[name][0] = bad
            with pytest.raises(error, match=r"\[0\]"):
                mxq.AdamW(**a)
        a = lists(eight=eight)
        n, dtype = a[name][0].numel(), a[name][0].dtype
        a[name][0] = on(1, n, dtype=dtype)
        with pytest.raises(ValueError, match="cuda:1"):
            mxq.AdamW(**a)
        a = lists(eight=eight)
        a[name].append(a[name][0])
        with pytest.raises(ValueError, match="params"):
            mxq.AdamW(**a)
    if eight:
        with pytest.raises(ValueError, match="belong together"):
            mxq.AdamW(**{**lists(), "v_scale": None})
    with pytest.raises(ValueError, match="no params"):
        mxq.AdamW([], [], [], [])
    with pytest.raises(ValueError, match="decay"):
        mxq.AdamW(**lists(), decay=[True])
    with pytest.raises(TypeError, match="copies"):
        mxq.AdamW(**lists(p=BF), copies=[on(0, 40, dtype=BF), None])


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
def test_tensors_of_a_set_that_share_memory_are_refused(stub, eight):
    """Two blocks would update the same elements at once."""
    for name in lists(eight=eight):
        if name in ("grads", "copies"):
            continue
        a = lists((300, 300), eight)
        a[name][1] = a[name][0]
        with pytest.raises(ValueError, match="shares memory"):
            mxq.AdamW(**a)
    flat = on(0, 600)
    a = lists((300, 300), eight)
    a["params"] = [flat[:300], flat[299:599]]
    with pytest.raises(ValueError, match=r"params\[1\] shares memory"):
        mxq.AdamW(**a)
    a["params"] = [flat[300:], flat[:300]]
    mxq.AdamW(**a)
    a["grads"][1] = a["grads"][0]  # only read
    mxq.AdamW(**a)
    a["grads"] = [flat[300:], flat[:300]]
    with pytest.raises(ValueError, match="shares memory"):
        mxq.AdamW(**a)


def test_an_update_set_steps_only_on_its_device_and_memory(stub, monkeypatch):
    a = lists()
    s = mxq.AdamW(**a)
    with pytest.raises(_Reached):
        s.step(1, 0.1)
    with pytest.raises(_Reached):
        s.step(on(0, 1, dtype=I64), on(0, 1), norm=on(0, 1), seed=-1)
    for bad in (dict(t=on(1, 1, dtype=I64)), dict(rate=on(1, 1)), dict(norm=on(1, 1))):
        with pytest.raises(ValueError, match="cuda:1"):
            s.step(**{**dict(t=1, rate=0.1), **bad})
    for bad in (dict(t=on(0, 1)), dict(rate=on(0, 1, dtype=BF)), dict(norm=on(0, 1, dtype=torch.float64))):
        with pytest.raises(TypeError):
            s.step(**{**dict(t=1, rate=0.1), **bad})
    for bad in (dict(t=on(0, 0, dtype=I64)), dict(rate=on(0, 0)), dict(norm=on(0, 0))):
        with pytest.raises(ValueError):
            s.step(**{**dict(t=1, rate=0.1), **bad})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="parameters are on cuda:0.*cuda:1"):
        s.step(1, 0.1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a["v_scale"][1].untyped_storage().resize_(1 << 16)
    with pytest.raises(ValueError, match="moved"):
        s.step(1, 0.1)


def test_the_norm_alone_is_of_the_current_device(stub, monkeypatch):
    s = mxq.GradientSet([on(0, 8), on(0, 4)])
    with pytest.raises(_Reached):
        s.norm(on(0, 1))
    with pytest.raises(ValueError, match="norm is on cuda:1"):
        s.norm(on(1, 1))
    with pytest.raises(TypeError, match="norm"):
        s.norm(on(0, 1, dtype=BF))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        s.norm(on(1, 1))
