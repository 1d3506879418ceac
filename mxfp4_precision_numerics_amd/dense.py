"""Layers and update that a low-precision recipe keeps out of FP8: the binding
of include/mxq_dense.h (same library, same manner as the package's other calls).

Linear layers with bias, activation and residual (linear), gated layers
(gated_linear), the gradients of both, and the AdamW step over any number of
tensors (AdamW), its moments in 32 bits or in 8.

Argument marshalling only, as training.py: outputs and workspaces are
preallocated tensors, every tensor's dtype, layout and extent are checked
before the library is called, and that it is on the current device; work goes
to ``stream`` (a handle of that device; default: the current one).
"""
import array
import ctypes

import mxfp4_precision_numerics_amd as _m

from . import training as _t

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4

_bound = None  # the library object whose signatures are set


def _lib():
    global _bound
    L = _m.lib()
    if _bound is not L:
        p, i64, i, d = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
        back = [p, i64, p, i64, p, i64, i, p, i64, p, i64, i64, i64, i64, p, i64, p, i, i64]
        for name, args, res in (
                ("mxq_linear_workspace", [i64, i64, i64, i], i64),
                ("mxq_linear", [p, i64, p, i64, p, i, p, i64, i64, i64, i64, p, i, i64, p, i64, p, i64, p], i),
                ("mxq_linear_backward", back + [p, i, p, i64, p], i),
                ("mxq_gated_linear_workspace", [i64, i64, i64, i], i64),
                ("mxq_gated_linear", [p, i64, p, i64, i, i64, i64, i64, p, i64, p, i64, p, i64, p], i),
                ("mxq_gated_linear_backward", back + [i, p, i64, p], i),
                ("mxq_adamw", [p, i64, p, i64, i, d, p, d, d, d, d, i64, p, p, d, ctypes.c_uint64, p], i),
                ("mxq_grad_norm", [p, i64, p, i64, p, p, p], i)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _bound = L
    return L


def _pitched(name, t, dtypes, rows, cols):
    """A matrix of just `cols` columns and at least `rows` rows, or None: (address, row pitch)."""
    if t is None:
        return None, 0
    if t.dtype in dtypes and t.dim() == 2:
        r, c = t.shape
        pitch, step = t.stride()
        if c == cols and r >= rows and (step == 1 or c == 1):
            return t.data_ptr(), pitch if rows > 1 else cols
    _t._two(name, t)
    _t._rows(name, t, dtypes, rows, cols)  # says what is wrong
    raise ValueError(f"{name} is {tuple(t.shape)}; the call has {cols} columns")


def _needed(name, t):
    if t is None:
        raise ValueError(f"{name} is required")


def _xw(x, w, D):
    """Sizes, addresses and row pitches of a call's x and w."""
    T, H = _t._two("x", x)
    N = _t._two("w", w)[0]
    px, ld_x = _pitched("x", x, D.bf16, T, H)
    pw, ld_w = _pitched("w", w, D.bf16, N, H)
    return T, H, N, px, ld_x, pw, ld_w


def _half(N):
    if N % 2:
        raise ValueError(f"w holds {N} rows; gate and up take as many each")
    return N // 2


def _on(stream, names, tensors):
    """Checked last: every tensor is on the current GPU; the stream that the call goes to."""
    D = _t._types()
    here = D.torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            _t._here(**dict(zip(names, tensors)))  # says which
    return _t._stream(stream, here)


_sizes = {}  # workspace bytes by a call's sizes: a function of them alone


def _workspace(fn, *sizes):
    n = _sizes.get((fn, sizes))
    if n is None:
        n = _t._size(fn, getattr(_lib(), fn + "_workspace")(*sizes))
        if len(_sizes) >= 4096:
            _sizes.clear()
        _sizes[fn, sizes] = n
    return n


def linear_workspace(tokens, hidden, features, backward=False):
    """Bytes of the workspace that linear (or, with ``backward``, linear_backward) takes."""
    return _workspace("mxq_linear", tokens, hidden, features, int(backward))


_LINEAR = "x", "w", "y", "bias", "residual", "z", "workspace"


def linear(x, w, y, bias=None, activation=ACT_NONE, residual=None, z=None, workspace=None, stream=None):
    """y = act(x w^T + bias) + residual (mxq_linear): ``x`` [tokens, hidden]
    and ``w`` [features, hidden] bfloat16, ``bias`` float32 [features], ``y``
    [tokens, features] bfloat16 or float32, ``residual`` like it (or ``y``
    itself).  ``z`` bfloat16 [tokens, features] receives what the activation
    is taken of, for linear_backward."""
    D = _t._types()
    L = _lib()
    T, H, N, px, ld_x, pw, ld_w = _xw(x, w, D)
    _needed("y", y)
    if residual is not None and residual.dtype != y.dtype:
        _t._same_type(y, residual=residual)
    py, ld_y = _pitched("y", y, D.floats, T, N)
    pr, ld_r = _pitched("residual", residual, D.floats, T, N)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    if bias is not None:
        _m._buf("bias", bias, D.f32, N)
    ws, n = _t._bytes("workspace", workspace, _workspace("mxq_linear", T, H, N, 0))
    on = _on(stream, _LINEAR, (x, w, y, bias, residual, z, workspace))
    _m._check("mxq_linear", L.mxq_linear(px, ld_x, pw, ld_w, _m._ptr(bias), activation, pr, ld_r, T, H, N, py,
                                         D.out[y.dtype], ld_y, pz, ld_z, ws, n, on))


_LINEAR_BACK = "x", "w", "dy", "dx", "dw", "dbias", "z", "add", "workspace"


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
    T, H, N, px, ld_x, pw, ld_w = _xw(x, w, D)
    _needed("dy", dy)
    if dx is None and dw is None and dbias is None:
        raise ValueError("dx, dw or dbias is required")
    if activation != ACT_NONE and z is None:
        raise ValueError("z is required with an activation")
    if add is not None and dx is None:
        raise ValueError("dx is required with add")
    py, ld_y = _pitched("dy", dy, D.bf16, T, N)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    pa, ld_a = _pitched("add", add, D.bf16, T, H)
    pdx, ld_dx = _pitched("dx", dx, D.bf16, T, H)
    pdw, ld_dw = _pitched("dw", dw, D.floats, N, H)
    if dbias is not None:
        _m._buf("dbias", dbias, D.f32, N)
    ws, n = _t._bytes("workspace", workspace, _workspace("mxq_linear", T, H, N, 1))
    on = _on(stream, _LINEAR_BACK, (x, w, dy, dx, dw, dbias, z, add, workspace))
    _m._check("mxq_linear_backward",
              L.mxq_linear_backward(px, ld_x, pw, ld_w, py, ld_y, activation, pz, ld_z, pa, ld_a, T, H, N, pdx, ld_dx,
                                    pdw, _m.OUT_F32 if dw is None else D.out[dw.dtype], ld_dw, _m._ptr(dbias),
                                    int(accumulate), ws, n, on))


def gated_linear_workspace(tokens, hidden, inter, backward=False):
    """Bytes of the workspace that gated_linear (or, with ``backward``, gated_linear_backward) takes."""
    return _workspace("mxq_gated_linear", tokens, hidden, inter, int(backward))


_GATED = "x", "w", "h", "z", "workspace"


def gated_linear(x, w, h, activation=ACT_SILU, z=None, workspace=None, stream=None):
    """h = act(x w_gate^T) * (x w_up^T) in one kernel (mxq_gated_linear): ``x``
    [tokens, hidden], ``w`` [2 inter, hidden] with the gate's rows first, ``h``
    [tokens, inter], all bfloat16.  ``z`` [tokens, 2 inter] receives gate and
    up, for gated_linear_backward."""
    D = _t._types()
    L = _lib()
    T, H, N, px, ld_x, pw, ld_w = _xw(x, w, D)
    inter = _half(N)
    _needed("h", h)
    ph, ld_h = _pitched("h", h, D.bf16, T, inter)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    ws, n = _t._bytes("workspace", workspace, _workspace("mxq_gated_linear", T, H, inter, 0))
    on = _on(stream, _GATED, (x, w, h, z, workspace))
    _m._check("mxq_gated_linear", L.mxq_gated_linear(px, ld_x, pw, ld_w, activation, T, H, inter, ph, ld_h, pz, ld_z, ws,
                                                     n, on))


_GATED_BACK = "x", "w", "dh", "dx", "dw", "z", "add", "workspace"


def gated_linear_backward(x, w, dh, dx=None, dw=None, activation=ACT_SILU, z=None, add=None, accumulate=False,
                          workspace=None, stream=None):
    """The gradients of gated_linear (mxq_gated_linear_backward) for ``dh``
    [tokens, inter] bfloat16; ``dx``, ``dw`` [2 inter, hidden], ``add`` and
    ``accumulate`` as linear_backward's.  ``z`` is what gated_linear left;
    None: gate and up are computed again."""
    D = _t._types()
    L = _lib()
    T, H, N, px, ld_x, pw, ld_w = _xw(x, w, D)
    inter = _half(N)
    _needed("dh", dh)
    if dx is None and dw is None:
        raise ValueError("dx or dw is required")
    if add is not None and dx is None:
        raise ValueError("dx is required with add")
    ph, ld_h = _pitched("dh", dh, D.bf16, T, inter)
    pz, ld_z = _pitched("z", z, D.bf16, T, N)
    pa, ld_a = _pitched("add", add, D.bf16, T, H)
    pdx, ld_dx = _pitched("dx", dx, D.bf16, T, H)
    pdw, ld_dw = _pitched("dw", dw, D.floats, N, H)
    ws, n = _t._bytes("workspace", workspace, _workspace("mxq_gated_linear", T, H, inter, 1))
    on = _on(stream, _GATED_BACK, (x, w, dh, dx, dw, z, add, workspace))
    _m._check("mxq_gated_linear_backward",
              L.mxq_gated_linear_backward(px, ld_x, pw, ld_w, ph, ld_h, activation, pz, ld_z, pa, ld_a, T, H, inter, pdx,
                                          ld_dx, pdw, _m.OUT_F32 if dw is None else D.out[dw.dtype], ld_dw,
                                          int(accumulate), ws, n, on))


class AdamW:
    """The tensors that one AdamW step covers: ``params`` and ``grads``, dense
    bfloat16 or float32 tensors of any size, the moments ``m`` and ``v`` of as
    many elements each, float32, or, with ``m_scale`` and ``v_scale``, 8 bits
    wide: uint8 codes (E4M3 and E5M2) and float32 scales, one for each BLOCK
    elements of a tensor and for what is left (zeros: moments of zero).
    ``copies``: bfloat16 tensors, or None, that receive the rounded values of
    float32 parameters.  ``decay``: for each tensor whether weight decay
    applies (default: to all).  Tensors share no memory (gradients may, with
    each other).

    It holds the tensors and the tables of their places on the device, and is
    built once for buffers that stay; step() takes what they hold then.
    Building one takes 4 to 6 us a tensor (157: 0.65 ms, in 8 bits 0.9) and
    waits for a copy, a step 7 to 35 us to call: gradients that are allocated
    anew at each step pay it each time, and are better kept.  As
    GradientSet, it covers the memory that they had when it was built, and
    keeps it: a tensor that is given other memory since is not followed and
    wants a new set; memory that was itself resized is refused by step().  It
    has to outlive the work that uses it."""

    CHUNK, BLOCK = 8192, 128  # MXQ_CLIP_CHUNK, MXQ_STATE_BLOCK

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, copies=None, decay=None):
        D = _t._types()
        torch = D.torch
        if (m_scale is None) != (v_scale is None):
            raise ValueError("m_scale and v_scale belong together")
        self._eight = m_scale is not None
        self.params = list(params)
        n = len(self.params)
        none = [None] * n
        self._lists = dict(params=self.params, grads=list(grads), m=list(m), v=list(v),
                           m_scale=list(m_scale) if self._eight else none,
                           v_scale=list(v_scale) if self._eight else none, copies=none if copies is None else list(copies))
        for name, ts in self._lists.items():
            if len(ts) != n:
                raise ValueError(f"{len(ts)} {name} for {n} params")
            if name != "copies" and (self._eight or not name.endswith("_scale")):
                for k, t in enumerate(ts):
                    _needed(f"{name}[{k}]", t)
        decay = [True] * n if decay is None else list(decay)
        if len(decay) != n:
            raise ValueError(f"{len(decay)} decay for {n} params")
        if n == 0:
            raise ValueError("no params")
        dev = self._device = self.params[0].get_device()
        if dev >= 0:
            _t._here(**{"params[0]": self.params[0]})
        rows, counts, first = array.array("q"), array.array("q"), 0
        src, chunk, f32, bf16 = D.src, self.CHUNK, torch.float32, torch.bfloat16
        state = torch.uint8 if self._eight else f32
        for k, (p, g, a, b, sa, sb, c) in enumerate(zip(*self._lists.values())):
            size = p.numel()
            ps, gs = src.get(p.dtype), src.get(g.dtype)
            fine = (ps is not None and gs is not None and a.dtype is b.dtype is state
                    and g.numel() == size == a.numel() == b.numel() and p.is_contiguous() and g.is_contiguous()
                    and a.is_contiguous() and b.is_contiguous()
                    and p.get_device() == g.get_device() == a.get_device() == b.get_device() == dev >= 0)
            at_sa = at_sb = at_c = 0
            if fine and self._eight:
                blocks = -(-size // self.BLOCK)
                fine = (sa.dtype is sb.dtype is f32 and sa.numel() == blocks == sb.numel() and sa.is_contiguous()
                        and sb.is_contiguous() and sa.get_device() == dev == sb.get_device())
                at_sa, at_sb = sa.data_ptr(), sb.data_ptr()
            if fine and c is not None:
                fine = (c.dtype is bf16 and p.dtype is f32 and c.numel() == size and c.is_contiguous()
                        and c.get_device() == dev)
                at_c = c.data_ptr()
            if not fine:
                self._refuse(k)
            rows.extend((p.data_ptr(), g.data_ptr(), a.data_ptr(), b.data_ptr(), at_sa, at_sb, at_c, size, first,
                         ps | gs << 32, 1 if decay[k] else 0))
            chunks = -(-size // chunk)
            counts.append(chunks)
            first += chunks
        self.chunks = first
        self._alone()
        every = [t for ts in self._lists.values() for t in ts if t is not None]
        self._storages = list(dict.fromkeys(map(torch.Tensor.untyped_storage, every)))
        self._places = self._at()
        # one copy to the device: the tensors' entries, then the chunks' tensors, two to a word
        of = torch.arange(n, dtype=torch.int32).repeat_interleave(torch.frombuffer(counts, dtype=torch.int64))
        if first % 2:
            of = torch.cat([of, of[:1]])
        self._tables = torch.cat([torch.frombuffer(rows, dtype=torch.int64), of.view(torch.int64)]).to(self.params[0].device)
        self._chunk_of = self._tables.data_ptr() + 8 * len(rows)
        self._streams = {_t._stream(None, dev)}  # that the allocator knows to use the tables

    _at = _t.GradientSet._at

    def _alone(self):
        """No tensor that a step writes shares memory with another one: two blocks would update it at once."""
        spans = sorted((t.data_ptr(), t.numel() * t.element_size(), name != "grads", name, k)
                       for name, ts in self._lists.items() for k, t in enumerate(ts) if t is not None and t.numel())
        written = end = 0  # where the tensors so far end
        for at, size, writes, name, k in spans:
            if at < (end if writes else written):
                raise ValueError(f"{name}[{k}] shares memory with another tensor of the set")
            end = max(end, at + size)
            if writes:
                written = max(written, at + size)

    def _refuse(self, k):
        """Say what is wrong with tensor k."""
        D = _t._types()
        t = {name: ts[k] for name, ts in self._lists.items()}
        state = D.u8 if self._eight else D.f32
        kinds = dict(params=D.floats, grads=D.floats, m=state, v=state, m_scale=D.f32, v_scale=D.f32, copies=D.bf16)
        size = t["params"].numel()
        for name, x in t.items():
            if x is None:
                continue
            _m._dtype(f"{name}[{k}]", x, kinds[name])
            if not x.is_contiguous():
                raise ValueError(f"{name}[{k}] must be contiguous")
            want = -(-size // self.BLOCK) if name in ("m_scale", "v_scale") else size
            if x.numel() != want:
                raise ValueError(f"{name}[{k}] holds {x.numel()} elements; params[{k}] of {size} has {want}")
        if t["copies"] is not None and t["params"].dtype != D.torch.float32:
            raise TypeError(f"copies[{k}]: params[{k}] is {t['params'].dtype}; a copy is of float32 parameters")
        _t._here(**{f"{name}[{k}]": x for name, x in t.items() if x is not None})

    def step(self, t, rate, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, norm=None, max_norm=1.0, seed=0,
             stream=None):
        """Step number ``t`` (from 1) at learning rate ``rate`` (mxq_adamw);
        either may be a tensor, int64 [1] and float32 [1], that the kernel
        reads: a captured step follows it.  ``norm`` float32 [1], as
        GradientSet.norm leaves it: the gradients are taken times min(1,
        max_norm / (norm + 1e-6)).  ``seed`` and ``t`` fix the 8-bit moments'
        rounding."""
        D = _t._types()
        L = _lib()
        tensors = {}
        if isinstance(t, D.torch.Tensor):
            _m._buf("t", t, D.i64, 1)
            tensors["t"] = t
        if isinstance(rate, D.torch.Tensor):
            _m._buf("rate", rate, D.f32, 1)
            tensors["rate"] = rate
        if norm is not None:
            _m._buf("norm", norm, D.f32, 1)
            tensors["norm"] = norm
        _t._here(**tensors)
        here = D.torch.cuda.current_device()
        if here != self._device:
            raise ValueError(f"the parameters are on cuda:{self._device}; the current device is cuda:{here}")
        if self._at() != self._places:
            raise ValueError("the tensors' memory was resized and has moved since the set was built")
        on = _t._stream(stream, here)
        if stream is None and on not in self._streams:  # else their memory could be taken while this call still runs
            self._tables.record_stream(D.torch.cuda.current_stream())
            self._streams.add(on)
        t_at, rate_at = tensors.get("t"), tensors.get("rate")
        _m._check("mxq_adamw",
                  L.mxq_adamw(self._tables.data_ptr(), len(self.params), self._chunk_of, self.chunks, int(self._eight),
                              0.0 if rate_at is not None else rate, _m._ptr(rate_at), betas[0], betas[1], eps,
                              weight_decay, 1 if t_at is not None else t, _m._ptr(t_at), _m._ptr(norm), max_norm,
                              seed & 0xFFFFFFFFFFFFFFFF, on))
