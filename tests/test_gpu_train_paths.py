"""GPU tests of the training-step operators on the paths that sizes, alignment
and places choose: losses on every tile, more places than a kernel holds at
once, scales at any address, gradient rows that move as vectors.

Tolerances are those of test_gpu_train_ops.py, from whose definitions in 64
bits the expected values come.
"""
import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from gpu_helpers import require_gpu
from test_gpu_train_ops import (BF, F32, H, HF, TINY, gen, lce_bounds, lce_case, lce_reference, routing, topk_back_reference,
                                topk_reference, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def forward(x, w, t):
    ws = torch.full((mxq.linear_cross_entropy_workspace(x.shape[0], x.shape[1], w.shape[0]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    loss, lse = (torch.full((x.shape[0],), 9.0, device="cuda") for _ in range(2))
    mxq.linear_cross_entropy(x, w, t, loss, lse, ws)
    return loss, lse


@pytest.mark.parametrize("T,Hd,V", [(2050, 512, 7717), (1025, 1024, 16001), (1100, 576, 30011), (2011, 2880, 9000),
                                    (4096, 512, 4096), (40000, 16, 4133), (70000, 16, 8133), (5, 520, 105001),
                                    (66, 1032, 130007), (127, 512, 31999), (100, 5120, 9001), (300, 264, 40001),
                                    (128, 4096, 32000)])
def test_losses_on_every_tile(T, Hd, V):
    """Targets among all words, the first and the last ones (a second launch's, a partial tile's) among them."""
    x, w, t, dloss = (a.cuda() for a in lce_case(T, Hd, V, 5))
    ends = torch.cat([torch.arange(3), V - 1 - torch.arange(300)]).cuda()
    at = torch.arange(0, T, 3, device="cuda")
    t[at] = ends[torch.arange(at.numel(), device="cuda") % ends.numel()]
    ref = lce_reference(x, w, t, dloss)
    e_lse, e_loss, _, _ = lce_bounds(ref, T, V, Hd)
    loss, lse = forward(x, w, t)
    within(lse, ref["lse"].cpu(), e_lse.cpu(), "lse")
    within(loss, ref["loss"].cpu(), torch.where(ref["ok"], e_loss, 0.0).cpu(), "loss")


@pytest.mark.parametrize("fmt", [mxq.E4M3, mxq.E5M2, mxq.E2M1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,C,k,E,G,at", [(5, 1024, 9, 12, 12, 0), (33, 2048, 9, 20, 11, 0), (7, 2048, 17, 40, 33, 0),
                                          (3, 1024, 64, 64, 64, 0), (9, 1024, 64, 80, 50, 0), (6, 1024, 65, 70, 66, 0),
                                          (21, 96, 11, 16, 13, 0), (2, 32, 100, 128, 90, 0), (19, 1024, 3, 8, 6, 1),
                                          (19, 2048, 8, 16, 9, 2), (11, 96, 11, 16, 13, 3)])
def test_dispatch_to_many_places_and_scales_at_any_address(T, C, k, E, G, at, dtype, fmt):
    pos, R = routing(T, k, E, G, T + C + k)
    R = max(R, 1) + 2
    x = torch.randn(T, C, generator=gen(C + k)) * 3
    x[:, 5] *= 1e4
    x[T - 1, 1] = float("nan")
    x = x.to(dtype).cuda()
    cpb = C // 2 if fmt == mxq.E2M1 else C
    u8 = lambda *s: torch.full(s, 0xA5, dtype=torch.uint8, device="cuda")
    q, qx, sx = u8(R, cpb), u8(T, cpb), u8(T, C // 32)
    held = u8(R * (C // 32) + 8)
    s = held[at:at + R * (C // 32)].view(R, C // 32)
    mxq.quantize_mx(x, fmt, qx, sx)
    mxq.moe_dispatch_mx(x, pos.cuda(), fmt, q, s)
    want_q, want_s = u8(R, cpb), u8(R, C // 32)
    for j in range(k):
        has = (pos[:, j] >= 0).nonzero()[:, 0].cuda()
        to = pos[:, j].cuda().long()[has]
        want_q[to], want_s[to] = qx[has], sx[has]
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    assert bool((held[:at] == 0xA5).all()) and bool((held[at + R * (C // 32):] == 0xA5).all())


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,pitch", [(9, 128, 4, 128), (300, 256, 8, 256), (5, 256, 10, 272), (18, 512, 16, 512),
                                         (7, 1024, 64, 1040), (6, 200, 5, 200), (4, 1008, 3, 1008), (3, 64, 8, 64)])
def test_topk_backward_of_rows_that_move_as_vectors(T, E, k, pitch, dtype, renorm):
    """Logits and gradients whose rows keep the alignment of a lane's run of experts."""
    g = gen(T + E + k)
    zc = torch.randn(T, E, generator=g).to(dtype)
    ids = topk_reference(zc, k, renorm)[0]
    gw = torch.randn(T, k, generator=g)
    z, wide = (torch.full((T, pitch), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    z[:, :E] = zc.cuda()
    mxq.moe_topk_backward(z[:, :E], ids.cuda(), gw.cuda(), wide[:, :E], renormalize=renorm)
    want = topk_back_reference(zc, ids, gw, renorm)
    top = gw.abs().amax(1, keepdim=True).double()
    p = torch.softmax(zc.double(), 1)
    p = p if not renorm else p / p.gather(1, ids.long()).sum(1, keepdim=True)
    within(wide[:, :E], want, (2 * E + 64) * HF * p * 2 * top + H[dtype] * want.abs() + TINY)
    assert bool((wide[:, E:] == 9.0).all())


def test_one_row_of_a_matrix_of_any_pitch():
    """One token: its row's stride to the next one says nothing (an odd one was refused for alignment)."""
    g = gen(61)
    wide = torch.randn(5, 67, generator=g).to(BF).cuda()
    x = wide[0:1, :64]
    dense = x.clone(memory_format=torch.contiguous_format)  # the quantizer wants a pitch
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    q, s, qx, sx = u8(1, 64), u8(1, 2), u8(1, 64), u8(1, 2)
    mxq.moe_dispatch_mx(x, pos, mxq.E4M3, q, s)
    mxq.quantize_mx(dense, mxq.E4M3, qx, sx)
    assert torch.equal(q, qx) and torch.equal(s, sx)
    y = torch.zeros(3, 67, dtype=BF, device="cuda")
    mxq.moe_combine(x, pos, y[:, :64])
    assert torch.equal(y[0, :64], x[0]) and not bool(y[1:].any()) and not bool(y[:, 64:].any())
    w = torch.randn(9, 64, generator=g).to(BF).cuda()
    t = torch.tensor([4], device="cuda")
    assert torch.equal(forward(x, w, t)[0], forward(dense, w, t)[0])
    ids, wt = torch.zeros(7, 1, dtype=torch.int32, device="cuda"), torch.zeros(7, 1, device="cuda")
    mxq.moe_topk(torch.ones(1, 7, device="cuda").t(), ids, wt)  # one expert: the column's stride
    assert not bool(ids.any()) and bool((wt == 1).all())


def test_a_gradient_set_keeps_its_memory_and_notices_that_it_moved():
    a, b = torch.full((5000,), 3.0, device="cuda"), torch.full((64,), 4.0, device="cuda", dtype=BF)
    norm = torch.zeros(1, device="cuda")
    s = mxq.GradientSet([a, b])
    place = a.data_ptr()
    a.data = torch.full((5000,), 5.0, device="cuda")  # no longer the set's
    others = [torch.full((5000,), 7.0, device="cuda") for _ in range(8)]
    assert place not in [o.data_ptr() for o in others]
    s.clip(1.0, norm)
    want = (5000 * 9.0 + 64 * 16.0) ** 0.5
    within(norm, torch.tensor([want], dtype=torch.float64), 2 * HF * want)
    assert bool((a == 5).all()) and all(bool((o == 7).all()) for o in others)
    b.untyped_storage().resize_(1 << 20)
    with pytest.raises(ValueError, match="moved"):
        s.clip(1.0, norm)
    mxq.GradientSet([a, b]).clip(0.0, norm)
    assert not bool(a.any())
