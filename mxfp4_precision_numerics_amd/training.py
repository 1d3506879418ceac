"""Training-step operators around the scaled GEMMs: the binding of
include/mxq_train.h (same library, same manner as the package's other calls).

The mixture-of-experts router (moe_topk, moe_sort), the movement of token
rows to and from their experts (moe_dispatch_mx, moe_combine), softmax cross
entropy against a vocabulary projection (linear_cross_entropy) and clipping
by the global gradient norm (GradientSet), with the gradients of each.

Argument marshalling only: outputs and workspaces are preallocated tensors,
every tensor's dtype, layout and extent are checked before the library is
called, and that it is on the current device; work goes to ``stream`` (a
handle of that device; default: the current one).
"""
import array
import ctypes

import mxfp4_precision_numerics_amd as _m

_bound = None  # the library object whose signatures are set


def _lib():
    global _bound
    L = _m.lib()
    if _bound is not L:
        p, i64, i, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        for name, args, res in (
                ("mxq_moe_topk", [p, i, i64, i64, i64, i64, i, p, p, p], i),
                ("mxq_moe_topk_backward", [p, i, i64, i64, i64, p, i64, i, p, p, i64, p], i),
                ("mxq_moe_sort_workspace", [i64, i64, i64], i64),
                ("mxq_moe_sort", [p, i64, i64, i64, p, p, p, p, i64, p], i),
                ("mxq_moe_dispatch_mx", [p, i, i64, i64, i64, p, i64, i, i64, p, p, p], i),
                ("mxq_moe_combine", [p, i, i64, i64, i64, p, i64, i64, p, p, i64, p], i),
                ("mxq_moe_combine_backward", [p, i, i64, i64, i64, p, i64, p, p, i64, i64, p, i64, p, p], i),
                ("mxq_linear_cross_entropy_workspace", [i64, i64, i64, i], i64),
                ("mxq_linear_cross_entropy", [p, i64, p, i64, p, i64, i64, i64, p, p, p, i64, p], i),
                ("mxq_linear_cross_entropy_backward",
                 [p, i64, p, i64, p, i64, i64, i64, p, p, p, i64, p, i64, p, i64, p], i),
                ("mxq_clip_grad_norm", [p, i64, p, i64, f, p, p, p], i)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _bound = L
    return L


class _Types:
    """The dtypes that the checks compare with, made on first use (the
    package imports torch only when it is called)."""

    def __init__(self):
        import torch
        self.torch = torch
        self.floats = (torch.bfloat16, torch.float32)
        self.bf16, self.f32, self.i32, self.i64, self.u8 = ((t,) for t in (torch.bfloat16, torch.float32, torch.int32,
                                                                           torch.int64, torch.uint8))
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # as the package's _stream, the device known
        self.src = {torch.float32: _m.SRC_F32, torch.bfloat16: _m.SRC_BF16}


_D = None


def _types():
    global _D
    if _D is None:
        _D = _Types()
    return _D


def _rows(name, t, dtypes, rows, cols):
    """A matrix view as _matrix wants it; the row pitch in elements.  Where a
    single row is addressed its stride says nothing and its length is taken;
    nor does a single column's."""
    if t.dtype in dtypes and t.dim() == 2:
        pitch, step = t.stride()
        r, c = t.shape
        if (step == 1 or c == 1) and r >= rows and c >= cols:
            return pitch if rows > 1 else cols
    _m._matrix(name, t, dtypes, rows, cols)  # says what is wrong
    return t.stride(0)


def _two(name, t):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def _same_type(x, **others):
    for name, t in others.items():
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {x.dtype}")


def _bytes(name, t, need):
    """A workspace of at least `need` bytes (may be None where none is needed)."""
    if t is None:
        if need > 0:
            raise ValueError(f"{name} is required")
        return None, 0
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    n = t.numel() * t.element_size()
    if n < need:
        raise ValueError(f"{name} holds {n} bytes; the call needs {need}")
    return t.data_ptr(), n


def _here(**tensors):
    """Checked last, as _on_gpu: every tensor is on the current GPU, whose
    stream the call goes to.  Returns its index."""
    here = None
    for name, t in tensors.items():
        if t is not None and t.get_device() != here:
            here = _first(name, t, here)
    return here


def _first(name, t, here):
    """The current device, for the first tensor; says what is wrong with any other."""
    if not t.is_cuda:
        _m._on_gpu(**{name: t})
    if here is None:
        here = _types().torch.cuda.current_device()
    if t.get_device() != here:
        raise ValueError(f"{name} is on cuda:{t.get_device()}; the current device is cuda:{here}")
    return here


def _stream(stream, here):
    """The handle of `stream`, by default the current one of the current device."""
    if stream is not None:
        return stream
    raw = _types().raw_stream
    return _m._stream(None) if raw is None else raw(here)


def _size(fn, n):
    _m._check(fn, min(n, 0))
    return n


def moe_topk(logits, ids, weights, renormalize=False, stream=None):
    """The topk = ids.shape[1] largest of each row of ``logits`` [tokens,
    experts] (bfloat16 or float32), equal ones by the lower expert, into
    ``ids`` int32 [tokens, topk], and their softmax ``weights`` float32
    [tokens, topk]: over all experts, or over the chosen ones
    (``renormalize``) (mxq_moe_topk)."""
    D = _types()
    L = _lib()
    T, E = _two("logits", logits)
    k = _two("ids", ids)[1]
    ld = _rows("logits", logits, D.floats, T, E)
    _m._buf("ids", ids, D.i32, T * k)
    _m._buf("weights", weights, D.f32, T * k)
    here = _here(logits=logits, ids=ids, weights=weights)
    _m._check("mxq_moe_topk", L.mxq_moe_topk(logits.data_ptr(), D.src[logits.dtype], T, E, ld, k, int(renormalize),
                                             ids.data_ptr(), weights.data_ptr(), _stream(stream, here)))


def moe_topk_backward(logits, ids, dweights, dlogits, renormalize=False, stream=None):
    """The gradient of moe_topk's weights: ``dweights`` float32 [tokens,
    topk] -> ``dlogits`` [tokens, experts] of the logits' type
    (mxq_moe_topk_backward)."""
    D = _types()
    L = _lib()
    T, E = _two("logits", logits)
    k = _two("ids", ids)[1]
    ld = _rows("logits", logits, D.floats, T, E)
    _same_type(logits, dlogits=dlogits)
    ld_d = _rows("dlogits", dlogits, D.floats, T, E)
    _m._buf("ids", ids, D.i32, T * k)
    _m._buf("dweights", dweights, D.f32, T * k)
    here = _here(logits=logits, ids=ids, dweights=dweights, dlogits=dlogits)
    _m._check("mxq_moe_topk_backward",
              L.mxq_moe_topk_backward(logits.data_ptr(), D.src[logits.dtype], T, E, ld, ids.data_ptr(), k,
                                      int(renormalize), dweights.data_ptr(), dlogits.data_ptr(), ld_d,
                                      _stream(stream, here)))


def moe_sort_workspace(tokens, topk, groups):
    """Bytes of the workspace that moe_sort takes."""
    return _size("mxq_moe_sort_workspace", _lib().mxq_moe_sort_workspace(tokens, topk, groups))


def moe_sort(ids, groups, off, src, pos, workspace=None, stream=None):
    """The assignments ``ids`` int32 [tokens, topk] in expert order
    (mxq_moe_sort): ``off`` int64 [groups + 1] as the grouped GEMMs take it,
    ``src`` int32 [tokens * topk] the token of each row (-1 past the last;
    may be None), ``pos`` int32 [tokens, topk] the row of each assignment
    (-1: its expert is not one of the ``groups``)."""
    D = _types()
    L = _lib()
    T, k = _two("ids", ids)
    _m._buf("ids", ids, D.i32, T * k)
    _m._buf("off", off, D.i64, groups + 1)
    if src is not None:
        _m._buf("src", src, D.i32, T * k)
    _m._buf("pos", pos, D.i32, T * k)
    ws, n = _bytes("workspace", workspace, _size("mxq_moe_sort", L.mxq_moe_sort_workspace(T, k, groups)))
    here = _here(ids=ids, off=off, src=src, pos=pos, workspace=workspace)
    _m._check("mxq_moe_sort", L.mxq_moe_sort(ids.data_ptr(), T, k, groups, off.data_ptr(), _m._ptr(src),
                                             pos.data_ptr(), ws, n, _stream(stream, here)))


def moe_dispatch_mx(x, pos, fmt, q, s, stream=None):
    """Rows of ``x`` [tokens, cols] (bfloat16 or float32), MX block-32
    quantized to ``fmt``, into the rows of ``q`` [rows, cols] (E2M1: [rows,
    cols/2]) and ``s`` [rows, cols/32] that ``pos`` int32 [tokens, topk]
    names (mxq_moe_dispatch_mx)."""
    D = _types()
    L = _lib()
    T, C = _two("x", x)
    k = _two("pos", pos)[1]
    R = _two("q", q)[0]
    ld = _rows("x", x, D.floats, T, C)
    _m._buf("pos", pos, D.i32, T * k)
    if pos.shape[0] < T:
        raise ValueError(f"pos holds {pos.shape[0]} tokens; the call addresses {T}")
    _m._buf("q", q, D.u8, R * _m._codes_per_row(fmt, C))
    _m._buf("s", s, D.u8, R * (C // 32))
    here = _here(x=x, pos=pos, q=q, s=s)
    _m._check("mxq_moe_dispatch_mx",
              L.mxq_moe_dispatch_mx(x.data_ptr(), D.src[x.dtype], T, C, ld, pos.data_ptr(), k, fmt, R, q.data_ptr(),
                                    s.data_ptr(), _stream(stream, here)))


def moe_combine(rows, pos, y, weights=None, stream=None):
    """y[t] = sum_j weights[t, j] * rows[pos[t, j]] (mxq_moe_combine);
    ``weights`` None: the plain sum, the gradient of a dispatch."""
    D = _types()
    L = _lib()
    R, C = _two("rows", rows)
    T, k = _two("pos", pos)
    ld_x = _rows("rows", rows, D.floats, R, C)
    _same_type(rows, y=y)
    ld_y = _rows("y", y, D.floats, T, C)
    _m._buf("pos", pos, D.i32, T * k)
    if weights is not None:
        _m._buf("weights", weights, D.f32, T * k)
    here = _here(rows=rows, pos=pos, y=y, weights=weights)
    _m._check("mxq_moe_combine",
              L.mxq_moe_combine(rows.data_ptr(), D.src[rows.dtype], R, C, ld_x, pos.data_ptr(), T, k,
                                _m._ptr(weights), y.data_ptr(), ld_y, _stream(stream, here)))


def moe_combine_backward(dy, pos, drows=None, weights=None, rows=None, dweights=None, stream=None):
    """The gradients of moe_combine (mxq_moe_combine_backward): ``drows``
    [rows, cols] (rows that ``pos`` names; the others are left alone) and
    ``dweights`` float32 [tokens, topk] (takes ``rows``); either may be
    None."""
    D = _types()
    L = _lib()
    T, C = _two("dy", dy)
    k = _two("pos", pos)[1]
    ld_dy = _rows("dy", dy, D.floats, T, C)
    if drows is None and dweights is None:
        raise ValueError("drows or dweights is required")
    if dweights is not None and rows is None:
        raise ValueError("rows is required with dweights")
    counts = [_two(n, t)[0] for n, t in (("drows", drows), ("rows", rows)) if t is not None]
    R = min(counts)
    _same_type(dy, drows=drows, rows=rows)
    ld_x = 0 if rows is None else _rows("rows", rows, D.floats, R, C)
    ld_dx = 0 if drows is None else _rows("drows", drows, D.floats, R, C)
    _m._buf("pos", pos, D.i32, T * k)
    if weights is not None:
        _m._buf("weights", weights, D.f32, T * k)
    if dweights is not None:
        _m._buf("dweights", dweights, D.f32, T * k)
    here = _here(dy=dy, pos=pos, drows=drows, weights=weights, rows=rows, dweights=dweights)
    _m._check("mxq_moe_combine_backward",
              L.mxq_moe_combine_backward(dy.data_ptr(), D.src[dy.dtype], T, C, ld_dy, pos.data_ptr(), k,
                                         _m._ptr(weights), _m._ptr(rows), ld_x, R, _m._ptr(drows), ld_dx,
                                         _m._ptr(dweights), _stream(stream, here)))


def linear_cross_entropy_workspace(tokens, hidden, vocab, backward=False):
    """Bytes of the workspace of linear_cross_entropy (and, with
    ``backward``, of its gradient too)."""
    return _size("mxq_linear_cross_entropy_workspace",
                 _lib().mxq_linear_cross_entropy_workspace(tokens, hidden, vocab, int(backward)))


def _lce(x, w, targets):
    D = _types()
    T, H = _two("x", x)
    V = _two("w", w)[0]
    ld_x = _rows("x", x, D.bf16, T, H)
    ld_w = _rows("w", w, D.bf16, V, H)
    if w.shape[1] != H:
        raise ValueError(f"w is {tuple(w.shape)}; x has {H} columns")
    _m._buf("targets", targets, D.i64, T)
    return T, H, V, ld_x, ld_w


def linear_cross_entropy(x, w, targets, loss, lse, workspace, stream=None):
    """Softmax cross entropy of ``x`` [tokens, hidden] against the projection
    ``w`` [vocab, hidden] (both bfloat16), the logits never stored
    (mxq_linear_cross_entropy): ``loss`` and ``lse`` float32 [tokens].  A
    target outside [0, vocab) is ignored: its loss is 0."""
    D = _types()
    L = _lib()
    T, H, V, ld_x, ld_w = _lce(x, w, targets)
    _m._buf("loss", loss, D.f32, T)
    _m._buf("lse", lse, D.f32, T)
    ws, n = _bytes("workspace", workspace, linear_cross_entropy_workspace(T, H, V))
    here = _here(x=x, w=w, targets=targets, loss=loss, lse=lse, workspace=workspace)
    _m._check("mxq_linear_cross_entropy",
              L.mxq_linear_cross_entropy(x.data_ptr(), ld_x, w.data_ptr(), ld_w, targets.data_ptr(), T, H, V,
                                         loss.data_ptr(), lse.data_ptr(), ws, n, _stream(stream, here)))


def linear_cross_entropy_backward(x, w, targets, lse, dloss, dx, dw, workspace, stream=None):
    """Its gradients from the forward call's ``lse`` and ``dloss`` float32
    [tokens] (mxq_linear_cross_entropy_backward): ``dx`` [tokens, hidden] and
    ``dw`` [vocab, hidden], bfloat16; either may be None."""
    D = _types()
    L = _lib()
    T, H, V, ld_x, ld_w = _lce(x, w, targets)
    _m._buf("lse", lse, D.f32, T)
    _m._buf("dloss", dloss, D.f32, T)
    if dx is None and dw is None:
        raise ValueError("dx or dw is required")
    ld_dx = 0 if dx is None else _rows("dx", dx, D.bf16, T, H)
    ld_dw = 0 if dw is None else _rows("dw", dw, D.bf16, V, H)
    ws, n = _bytes("workspace", workspace, linear_cross_entropy_workspace(T, H, V, True))
    here = _here(x=x, w=w, targets=targets, lse=lse, dloss=dloss, dx=dx, dw=dw, workspace=workspace)
    _m._check("mxq_linear_cross_entropy_backward",
              L.mxq_linear_cross_entropy_backward(x.data_ptr(), ld_x, w.data_ptr(), ld_w, targets.data_ptr(), T, H,
                                                  V, lse.data_ptr(), dloss.data_ptr(), _m._ptr(dx), ld_dx,
                                                  _m._ptr(dw), ld_dw, ws, n, _stream(stream, here)))


class GradientSet:
    """The gradients that one clipping covers: ``grads``, dense bfloat16 or
    float32 tensors of any size, and ``out``, tensors like them that receive
    the clipped values (default: the gradients themselves).  It holds the
    tensors and the tables of their places and chunks on the device, and is
    built once for buffers that stay; clip() takes what they hold then.  It
    covers the memory that they had when it was built, and keeps it: a tensor
    that is given other memory (.data, set_) or another shape since is not
    followed and wants a new set, as do gradients that are allocated anew at
    each step; memory that was itself resized is refused by clip().  Like any
    tensor it has to outlive the work that uses it: calls on a ``stream``
    given by handle, and the replays of a graph that a call was captured in.
    Calls on several streams share its scratch memory and must not overlap."""

    CHUNK, PARTS = 8192, 2048  # MXQ_CLIP_CHUNK, MXQ_CLIP_PARTS

    def __init__(self, grads, out=None):
        D = _types()
        torch = D.torch
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"{len(self.out)} outputs for {len(self.grads)} gradients")
        if not self.grads:
            raise ValueError("no gradients")
        dev = self._device = self.grads[0].get_device()
        if dev >= 0:
            _here(**{"grads[0]": self.grads[0]})
        rows, counts, first = array.array("q"), array.array("q"), 0
        src, chunk = D.src, self.CHUNK
        for n, (g, o) in enumerate(zip(self.grads, self.out)):
            size = g.numel()
            kind = src.get(g.dtype)
            place = g.data_ptr()
            to = place
            fine = kind is not None and g.is_contiguous() and g.get_device() == dev >= 0
            if fine and o is not g:
                to = o.data_ptr()
                fine = src.get(o.dtype) == kind and o.is_contiguous() and o.numel() == size and o.get_device() == dev
            if not fine:
                self._refuse(n, g, o)
            chunks = -(-size // chunk)
            rows.extend((place, to, size, kind, first))
            counts.append(chunks)
            first += chunks
        self.chunks = first
        lists = (self.grads,) if self.out is self.grads else (self.grads, self.out)
        self._storages = list(dict.fromkeys(s for t in lists for s in map(torch.Tensor.untyped_storage, t)))
        self._places = self._at()
        # one copy to the device: the tensors' entries, then the chunks' tensors, two to a word
        of = torch.arange(len(counts), dtype=torch.int32).repeat_interleave(torch.frombuffer(counts, dtype=torch.int64))
        if first % 2:
            of = torch.cat([of, of[:1]])
        self._tables = torch.cat([torch.frombuffer(rows, dtype=torch.int64), of.view(torch.int64)]).to(self.grads[0].device)
        self._chunk_of = self._tables.data_ptr() + 8 * len(rows)
        self._parts = torch.empty(self.PARTS, dtype=torch.float64, device=self.grads[0].device)
        self._streams = {_stream(None, dev)}  # that the allocator knows to use the tables

    def _at(self):
        """Where the memory is: an address for each storage (0.03 us), not for each tensor."""
        return list(map(_types().torch.UntypedStorage.data_ptr, self._storages))

    def _refuse(self, n, g, o):
        """Say what is wrong with gradient n."""
        D = _types()
        _m._dtype(f"grads[{n}]", g, D.floats)
        _same_type(g, **{f"out[{n}]": o})
        for name, t in ((f"grads[{n}]", g), (f"out[{n}]", o)):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if o.numel() != g.numel():
            raise ValueError(f"out[{n}] holds {o.numel()} elements, grads[{n}] {g.numel()}")
        _here(**{f"grads[{n}]": g, f"out[{n}]": o})

    def clip(self, max_norm, norm, stream=None):
        """``norm`` float32 [1] = the global 2-norm before clipping; out =
        grads * min(1, max_norm / (norm + 1e-6)) (mxq_clip_grad_norm)."""
        D = _types()
        L = _lib()
        _m._buf("norm", norm, D.f32, 1)
        here = _here(norm=norm)
        if here != self._device:
            raise ValueError(f"the gradients are on cuda:{self._device}; the current device is cuda:{here}")
        if self._at() != self._places:
            raise ValueError("the gradients' or outputs' memory was resized and has moved since the set was built")
        on = _stream(stream, here)
        if stream is None and on not in self._streams:  # else their memory could be taken while this call still runs
            for t in (self._tables, self._parts):
                t.record_stream(D.torch.cuda.current_stream())
            self._streams.add(on)
        _m._check("mxq_clip_grad_norm",
                  L.mxq_clip_grad_norm(self._tables.data_ptr(), len(self.grads), self._chunk_of, self.chunks,
                                       max_norm, norm.data_ptr(), self._parts.data_ptr(), on))
