"""Layers and update that a low-precision recipe keeps out of FP8: the binding
of include/mxq_dense.h (same library, same manner as the package's other calls).

Linear layers with bias, activation and residual (linear), gated layers
(gated_linear) and the gradients of both.

Argument marshalling only, as training.py: outputs and workspaces are
preallocated tensors, every tensor's dtype, layout and extent are checked
before the library is called, and that it is on the current device; work goes
to ``stream`` (a handle of that device; default: the current one).
"""
import ctypes

import mxfp4_precision_numerics_amd as _m

from . import training as _t

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4

_bound = None  # the library object whose signatures are set


def _lib():
    global _bound
    L = _m.lib()
    if _bound is not L:
        p, i64, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        back = [p, i64, p, i64, p, i64, i, p, i64, p, i64, i64, i64, i64, p, i64, p, i, i64]
        for name, args, res in (
                ("mxq_linear_workspace", [i64, i64, i64, i], i64),
                ("mxq_linear", [p, i64, p, i64, p, i, p, i64, i64, i64, i64, p, i, i64, p, i64, p, i64, p], i),
                ("mxq_linear_backward", back + [p, i, p, i64, p], i),
                ("mxq_gated_linear_workspace", [i64, i64, i64, i], i64),
                ("mxq_gated_linear", [p, i64, p, i64, i, i64, i64, i64, p, i64, p, i64, p, i64, p], i),
                ("mxq_gated_linear_backward", back + [i, p, i64, p], i)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _bound = L
    return L


def _pitched(name, t, dtypes, rows, cols):
    """A matrix of just `cols` columns and at least `rows` rows, or None: (address, row pitch)."""
    if t is None:
        return None, 0
    ld = _t._rows(name, t, dtypes, rows, cols)
    if t.shape[1] != cols:
        raise ValueError(f"{name} is {tuple(t.shape)}; the call has {cols} columns")
    return t.data_ptr(), ld


def _out_of(t):
    return _m.OUT_F32 if t is None or t.dtype == _t._types().torch.float32 else _m.OUT_BF16


def _xw(x, w, D):
    T, H = _t._two("x", x)
    N = _t._two("w", w)[0]
    ld_x = _t._rows("x", x, D.bf16, T, H)
    ld_w = _t._rows("w", w, D.bf16, N, H)
    if w.shape[1] != H:
        raise ValueError(f"w is {tuple(w.shape)}; x has {H} columns")
    return T, H, N, ld_x, ld_w


def _half(w):
    if w.shape[0] % 2:
        raise ValueError(f"w holds {w.shape[0]} rows; gate and up take as many each")
    return w.shape[0] // 2


def linear_workspace(tokens, hidden, features, backward=False):
    """Bytes of the workspace that linear (or, with ``backward``, linear_backward) takes."""
    return _t._size("mxq_linear_workspace", _lib().mxq_linear_workspace(tokens, hidden, features, int(backward)))


def linear(x, w, y, bias=None, activation=ACT_NONE, residual=None, z=None, workspace=None, stream=None):
    """y = act(x w^T + bias) + residual (mxq_linear): ``x`` [tokens, hidden]
    and ``w`` [features, hidden] bfloat16, ``bias`` float32 [features], ``y``
    [tokens, features] bfloat16 or float32, ``residual`` like it (or ``y``
    itself).  ``z`` bfloat16 [tokens, features] receives what the activation
    is taken of, for linear_backward."""
    D = _t._types()
    L = _lib()
    T, H, N, ld_x, ld_w = _xw(x, w, D)
    _t._two("y", y)
    _t._same_type(y, residual=residual)
    py, ld_y = _pitched("y", y, D.floats, T, N)
    pr, ld_r = _pitched("residual", residual, D.floats, T, N)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    if bias is not None:
        _m._buf("bias", bias, D.f32, N)
    ws, n = _t._bytes("workspace", workspace, linear_workspace(T, H, N))
    here = _t._here(x=x, w=w, y=y, bias=bias, residual=residual, z=z, workspace=workspace)
    _m._check("mxq_linear",
              L.mxq_linear(x.data_ptr(), ld_x, w.data_ptr(), ld_w, _m._ptr(bias), activation, pr, ld_r, T, H, N, py,
                           _out_of(y), ld_y, pz, ld_z, ws, n, _t._stream(stream, here)))


def linear_backward(x, w, dy, dx=None, dw=None, dbias=None, activation=ACT_NONE, z=None, add=None, accumulate=False,
                    workspace=None, stream=None):
    """The gradients of linear (mxq_linear_backward) for ``dy`` [tokens,
    features] bfloat16: ``dx`` [tokens, hidden] bfloat16, joined by ``add``
    (a skip connection's gradient; may be ``dx`` itself), ``dw`` [features,
    hidden] bfloat16 or float32, ``dbias`` float32 [features]; each may be
    None.  ``accumulate``: dw and dbias are added to what they hold.  ``z`` is
    what linear left (with an activation)."""
    D = _t._types()
    L = _lib()
    T, H, N, ld_x, ld_w = _xw(x, w, D)
    _t._two("dy", dy)
    if dx is None and dw is None and dbias is None:
        raise ValueError("dx, dw or dbias is required")
    if activation != ACT_NONE and z is None:
        raise ValueError("z is required with an activation")
    if add is not None and dx is None:
        raise ValueError("dx is required with add")
    pd, ld_dy = _pitched("dy", dy, D.bf16, T, N)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    pa, ld_a = _pitched("add", add, D.bf16, T, H)
    px, ld_dx = _pitched("dx", dx, D.bf16, T, H)
    pw, ld_dw = _pitched("dw", dw, D.floats, N, H)
    if dbias is not None:
        _m._buf("dbias", dbias, D.f32, N)
    ws, n = _t._bytes("workspace", workspace, linear_workspace(T, H, N, True) if T else 0)
    here = _t._here(x=x, w=w, dy=dy, dx=dx, dw=dw, dbias=dbias, z=z, add=add, workspace=workspace)
    _m._check("mxq_linear_backward",
              L.mxq_linear_backward(x.data_ptr(), ld_x, w.data_ptr(), ld_w, pd, ld_dy, activation, pz, ld_z, pa, ld_a, T,
                                    H, N, px, ld_dx, pw, _out_of(dw), ld_dw, _m._ptr(dbias), int(accumulate), ws, n,
                                    _t._stream(stream, here)))


def gated_linear_workspace(tokens, hidden, inter, backward=False):
    """Bytes of the workspace that gated_linear (or, with ``backward``, gated_linear_backward) takes."""
    return _t._size("mxq_gated_linear_workspace",
                    _lib().mxq_gated_linear_workspace(tokens, hidden, inter, int(backward)))


def gated_linear(x, w, h, activation=ACT_SILU, z=None, workspace=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) in one kernel (mxq_gated_linear): ``x``
    [tokens, hidden], ``w`` [2 inter, hidden] with the gate's rows first, ``h``
    [tokens, inter], all bfloat16.  ``z`` [tokens, 2 inter] receives gate and
    up, for gated_linear_backward."""
    D = _t._types()
    L = _lib()
    T, H, N, ld_x, ld_w = _xw(x, w, D)
    inter = _half(w)
    _t._two("h", h)
    ph, ld_h = _pitched("h", h, D.bf16, T, inter)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    ws, n = _t._bytes("workspace", workspace, gated_linear_workspace(T, H, inter))
    here = _t._here(x=x, w=w, h=h, z=z, workspace=workspace)
    _m._check("mxq_gated_linear",
              L.mxq_gated_linear(x.data_ptr(), ld_x, w.data_ptr(), ld_w, activation, T, H, inter, ph, ld_h, pz, ld_z,
                                 ws, n, _t._stream(stream, here)))


def gated_linear_backward(x, w, dh, dx=None, dw=None, activation=ACT_SILU, z=None, add=None, accumulate=False,
                          workspace=None, stream=None):
    """The gradients of gated_linear (mxq_gated_linear_backward) for ``dh``
    [tokens, inter] bfloat16; ``dx``, ``dw`` [2 inter, hidden], ``add`` and
    ``accumulate`` as linear_backward's.  ``z`` is what gated_linear left;
    None: gate and up are computed again."""
    D = _t._types()
    L = _lib()
    T, H, N, ld_x, ld_w = _xw(x, w, D)
    inter = _half(w)
    _t._two("dh", dh)
    if dx is None and dw is None:
        raise ValueError("dx or dw is required")
    if add is not None and dx is None:
        raise ValueError("dx is required with add")
    pd, ld_dh = _pitched("dh", dh, D.bf16, T, inter)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    pa, ld_a = _pitched("add", add, D.bf16, T, H)
    px, ld_dx = _pitched("dx", dx, D.bf16, T, H)
    pw, ld_dw = _pitched("dw", dw, D.floats, N, H)
    ws, n = _t._bytes("workspace", workspace, gated_linear_workspace(T, H, inter, True) if T else 0)
    here = _t._here(x=x, w=w, dh=dh, dx=dx, dw=dw, z=z, add=add, workspace=workspace)
    _m._check("mxq_gated_linear_backward",
              L.mxq_gated_linear_backward(x.data_ptr(), ld_x, w.data_ptr(), ld_w, pd, ld_dh, activation, pz, ld_z, pa,
                                          ld_a, T, H, inter, px, ld_dx, pw, _out_of(dw), ld_dw, int(accumulate), ws, n,
                                          _t._stream(stream, here)))
