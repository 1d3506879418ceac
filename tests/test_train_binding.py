"""What the binding of the training-step operators passes on (CPU checks): row
pitches of views of which a stride says nothing, and no tensor of another GPU than the current one."""
import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from mxfp4_precision_numerics_amd import training

F = (torch.float32,)


def pitch(t, rows, cols):
    return training._rows("t", t, F, rows, cols)


def test_a_single_rows_stride_says_nothing():
    wide = torch.zeros(9, 33)
    assert pitch(wide[4:5, :32], 1, 32) == 32  # 33 would be refused for alignment
    assert pitch(wide[:, :32], 1, 32) == 32  # one row is addressed
    assert pitch(wide[:0, :32], 0, 32) == 32
    assert pitch(wide[::2, :32], 5, 32) == 66
    assert pitch(wide[:2, :32], 2, 32) == 33


def test_a_single_columns_stride_says_nothing():
    t = torch.zeros(1, 7).t()
    assert t.is_contiguous() and t.stride(1) != 1
    assert pitch(t, 7, 1) == 1
    with pytest.raises(ValueError, match="unit column stride"):
        pitch(torch.zeros(2, 7).t(), 7, 2)


@pytest.mark.parametrize("t,rows,cols", [(torch.zeros(3, 32), 4, 32), (torch.zeros(1, 31), 1, 32), (torch.zeros(0, 32), 1, 32)])
def test_a_view_too_small_is_refused(t, rows, cols):
    with pytest.raises(ValueError, match="the call addresses"):
        pitch(t, rows, cols)


# Tensors of GPUs that are not there: their device is all that the checks look at.
class On(torch.Tensor):
    """A host tensor that gives itself out as one of GPU `gpu`."""
    is_cuda, gpu = True, 0  # views are of GPU 0

    def get_device(self):
        return self.gpu


def on(gpu, *shape, dtype=torch.float32):
    t = torch.Tensor._make_subclass(On, torch.zeros(shape, dtype=dtype))
    t.gpu = gpu
    return t


BF, I32, I64, U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8


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
def two_gpus(monkeypatch):
    """GPU 0 is the current one."""
    monkeypatch.setattr(mxq, "_lib", _Library())
    monkeypatch.setattr(training, "_bound", mxq._lib)
    monkeypatch.setattr(training, "_stream", lambda s, here: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


# (call, its tensors: name, shape, dtype) - all on one device but for the one under test
CALLS = {
    "moe_topk": [("logits", (4, 16), BF), ("ids", (4, 2), I32), ("weights", (4, 2), torch.float32)],
    "moe_topk_backward": [("logits", (4, 16), BF), ("ids", (4, 2), I32), ("dweights", (4, 2), torch.float32),
                          ("dlogits", (4, 16), BF)],
    "moe_sort": [("ids", (4, 2), I32), ("off", (9,), I64), ("src", (8,), I32), ("pos", (4, 2), I32), ("workspace", (16,), U8)],
    "moe_dispatch_mx": [("x", (4, 64), BF), ("pos", (4, 2), I32), ("q", (8, 64), U8), ("s", (8, 2), U8)],
    "moe_combine": [("rows", (8, 64), BF), ("pos", (4, 2), I32), ("y", (4, 64), BF), ("weights", (4, 2), torch.float32)],
    "moe_combine_backward": [("dy", (4, 64), BF), ("pos", (4, 2), I32), ("drows", (8, 64), BF),
                             ("weights", (4, 2), torch.float32), ("rows", (8, 64), BF), ("dweights", (4, 2), torch.float32)],
    "linear_cross_entropy": [("x", (4, 64), BF), ("w", (9, 64), BF), ("targets", (4,), I64), ("loss", (4,), torch.float32),
                             ("lse", (4,), torch.float32), ("workspace", (16,), U8)],
    "linear_cross_entropy_backward": [("x", (4, 64), BF), ("w", (9, 64), BF), ("targets", (4,), I64),
                                      ("lse", (4,), torch.float32), ("dloss", (4,), torch.float32), ("dx", (4, 64), BF),
                                      ("dw", (9, 64), BF), ("workspace", (16,), U8)],
}
MORE = {"moe_sort": dict(groups=8), "moe_dispatch_mx": dict(fmt=0)}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(two_gpus, name):
    def call(where):
        getattr(mxq, name)(**{n: on(where(n), *s, dtype=d) for n, s, d in CALLS[name]}, **MORE.get(name, {}))
    with pytest.raises(_Reached):
        call(lambda n: 0)
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):  # whose stream the call would not go to
        call(lambda n: 1)
    for odd, _, _ in CALLS[name]:
        with pytest.raises(ValueError, match=f"^{odd} is on cuda:1"):
            call(lambda n: int(n == odd))


def test_a_gradient_set_is_of_the_current_device(two_gpus, monkeypatch):
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        mxq.GradientSet([on(1, 8), on(1, 4)])
    with pytest.raises(ValueError, match="cuda:1"):
        mxq.GradientSet([on(0, 8), on(1, 4)])
    with pytest.raises(ValueError, match="cuda:1"):
        mxq.GradientSet([on(0, 8)], [on(1, 8)])
    s = mxq.GradientSet.__new__(mxq.GradientSet)  # as built on GPU 0, without its tables
    s.grads = s.out = [on(0, 8)]
    s._tables, s._parts, s._chunk_of, s.chunks, s._streams, s._device = on(0, 4), on(0, 4), 0, 1, {0}, 0
    with pytest.raises(ValueError, match="norm is on cuda:1"):
        s.clip(1.0, on(1, 1))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="norm is on cuda:0.*cuda:1"):
        s.clip(1.0, on(0, 1))
    with pytest.raises(ValueError, match="gradients are on cuda:0.*cuda:1"):
        s.clip(1.0, on(1, 1))


def test_a_gradient_set_whose_memory_moved_is_refused(two_gpus):
    """The tables hold addresses: memory that went elsewhere since is not read or written at the old ones."""
    for move in (lambda t: t.untyped_storage().resize_(0), lambda t: t.untyped_storage().resize_(1 << 16),
                 lambda t: t.resize_(1 << 14)):
        for which in range(4):
            flat = on(0, 24)
            a, b, c, d = on(0, 8), on(0, 5, dtype=BF), flat, on(0, 5, dtype=BF)
            s = mxq.GradientSet([a, b], [c[8:16], d])
            with pytest.raises(_Reached):
                s.clip(1.0, on(0, 1))
            move((a, b, c, d)[which])
            with pytest.raises(ValueError, match="moved"):
                s.clip(1.0, on(0, 1))


def test_a_gradient_set_keeps_the_memory_that_it_was_built_for(two_gpus):
    """A tensor that is given other memory (.data, set_) does not free what the tables point at."""
    a, b = on(0, 1 << 16), on(0, 1 << 16)
    places = [a.data_ptr(), b.data_ptr()]
    kept = [a.untyped_storage()._weak_ref(), b.untyped_storage()._weak_ref()]
    s = mxq.GradientSet([a, b])
    a.data = torch.zeros(1 << 16)
    b.set_(torch.zeros(1 << 16))
    assert a.data_ptr() != places[0] and b.data_ptr() != places[1]
    assert not any(torch.UntypedStorage._expired(k) for k in kept)
    with pytest.raises(_Reached):
        s.clip(1.0, on(0, 1))
    del s
    assert all(torch.UntypedStorage._expired(k) for k in kept)
    for k in kept:
        torch.UntypedStorage._free_weak_ref(k)
