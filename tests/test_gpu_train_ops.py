"""GPU tests of the training-step operators against their definitions in 64
bits, at the sizes, masks and strides where they can go wrong.

Tolerances.  A rounding to a type is off by at most half a step, H(t) =
finfo(t).eps / 2 relative (bf16 2^-8, fp32 2^-24); a binary32 sum of n terms
by (n + 1) H(fp32) times the sum of the terms' magnitudes (any order); the
binary32 exp and log by 4 H(fp32) relative, the fast exp by (2 + |argument|)
* 2 H(fp32) (the argument is scaled by log2 e first).  Each check states the
terms that it counts.  Whole numbers and quantized codes are equal.
"""
import numpy as np
import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HF = 2.0 ** -24
H = {BF: 2.0 ** -8, F32: HF}
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, bound, what=""):
    got, want = got.detach().cpu().double(), want.double()
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: NaN in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~nan & ~inf
    err, b = (got - want).abs()[ok], torch.as_tensor(bound, dtype=F64).expand_as(want)[ok]
    assert bool((err <= b).all()), f"{what}: off by {float((err / b.clamp(min=1e-300)).max()):.3g} times the bound"


# ------------------------------------------------------------------ router

def topk_reference(zc, k, renorm):
    """The definition in 64 bits on the CPU: ids by (value descending, index)."""
    z = zc.double().numpy()
    key = np.where(np.isnan(z), np.inf, z)
    rank = np.argsort(-key, axis=1, kind="stable")
    for t in np.nonzero(np.isnan(z).any(axis=1))[0]:  # NaN above +inf
        rank[t] = sorted(range(z.shape[1]), key=lambda e: (not np.isnan(z[t, e]), -key[t, e], e))
    ids = rank[:, :k]
    top = torch.from_numpy(np.take_along_axis(z, rank[:, :1], 1))
    e = (zc.double() - top).exp()
    pick = e.gather(1, torch.from_numpy(ids.astype(np.int64)))
    return torch.from_numpy(ids.astype(np.int32)), pick / (pick if renorm else e).sum(1, keepdim=True)


def gpu_topk(z, k, renorm):
    ids = torch.full((z.shape[0], k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((z.shape[0], k), -7.0, device="cuda")
    mxq.moe_topk(z, ids, w, renormalize=renorm)
    return ids, w


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 4, 4), (3, 63, 7), (16, 64, 8), (7, 65, 1), (33, 129, 10), (257, 256, 8),
                                   (9, 513, 64), (2, 1024, 6), (1001, 300, 3)])
def test_topk(T, E, k, dtype, renorm):
    zc = (torch.randn(T, E, generator=gen(T * E + k)) * 2).to(dtype)
    ids, w = gpu_topk(zc.cuda(), k, renorm)
    want_ids, want = topk_reference(zc, k, renorm)
    assert torch.equal(ids.cpu(), want_ids)
    # exp of the pick and of each summand (argument rounded: |z - m| H more), the sum, the quotient
    rel = (8 + E + 2 * float(zc.float().max() - zc.float().min())) * HF
    within(w, want, rel * want + TINY)


def test_topk_ties_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    zc = torch.tensor([[1.0, 2.0, 2.0, 2.0, 0.0], [0.0, -0.0, 0.0, -0.0, 0.0], [-inf, -inf, 1.0, -inf, -inf],
                       [-inf] * 5, [inf, 1.0, inf, 0.0, -inf], [1.0, nan, 3.0, nan, inf],
                       [3e38, -3e38, 3e38, 1.0, 0.0]])
    ids, w = gpu_topk(zc.cuda(), 4, False)
    want_ids, want = topk_reference(zc, 4, False)
    assert torch.equal(ids.cpu(), want_ids)
    within(w, want, 16 * HF * want.nan_to_num() + TINY)
    ids, w = gpu_topk(zc[:1].expand(1, 5).to(BF).cuda(), 3, True)
    assert ids.tolist() == [[1, 2, 3]]


def test_topk_row_pitch_and_offset():
    big = torch.randn(20, 301, generator=gen(5))
    zc = big[:, 1:260]
    ids, w = gpu_topk(big.cuda()[:, 1:260], 8, True)
    want_ids, want = topk_reference(zc, 8, True)
    assert torch.equal(ids.cpu(), want_ids)
    within(w, want, 300 * HF * want + TINY)


def topk_back_reference(z, ids, g, renorm):
    z = z.double().clone().requires_grad_()
    p = torch.softmax(z, 1).gather(1, ids.long())
    (p / p.sum(1, keepdim=True) if renorm else p).backward(g.double())
    return z.grad


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (6, 4, 2), (17, 64, 8), (5, 257, 10), (300, 256, 8), (3, 1024, 64)])
def test_topk_backward(T, E, k, dtype, renorm):
    g = gen(T + E + k)
    zc = torch.randn(T, E, generator=g).to(dtype)
    ids = topk_reference(zc, k, renorm)[0]
    gw = torch.randn(T, k, generator=g)
    wide = torch.full((T, E + 3), 9.0, dtype=dtype, device="cuda")
    mxq.moe_topk_backward(zc.cuda(), ids.cuda(), gw.cuda(), wide[:, :E], renormalize=renorm)
    want = topk_back_reference(zc, ids, gw, renorm)
    # p (E + 16 roundings), the dot product, their difference; then the output's half step
    top = gw.abs().amax(1, keepdim=True).double()
    p = torch.softmax(zc.double(), 1)
    p = p if not renorm else p / p.gather(1, ids.long()).sum(1, keepdim=True)
    within(wide[:, :E], want, (2 * E + 64) * HF * p * 2 * top + H[dtype] * want.abs() + TINY)
    assert bool((wide[:, E:] == 9.0).all())


def test_topk_backward_against_differences():
    g = gen(11)
    T, E, k = 4, 32, 4
    zc = torch.randn(T, E, generator=g).double()
    ids = topk_reference(zc.float(), k, True)[0].long()
    gw = torch.randn(T, k, generator=g).double()
    f = lambda z: (torch.softmax(z, 1).gather(1, ids) / torch.softmax(z, 1).gather(1, ids).sum(1, keepdim=True) * gw).sum()
    dz = torch.empty(T, E, device="cuda")
    mxq.moe_topk_backward(zc.float().cuda(), ids.int().cuda(), gw.float().cuda(), dz, renormalize=True)
    d, h = torch.randn(T, E, generator=g).double(), 1e-5
    slope = (f(zc.float().double() + h * d) - f(zc.float().double() - h * d)) / (2 * h)
    # the differences' own error: h^2 of a third derivative of order |d|^3 |gw|
    assert abs(float((dz.cpu().double() * d).sum() - slope)) < 1e-5 * float(d.abs().sum())


def test_topk_backward_ids_out_of_range_add_nothing():
    zc = torch.randn(2, 16, generator=gen(1)).cuda()
    ids = torch.tensor([[3, -1], [16, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    gw, dz = torch.ones(2, 2, device="cuda"), torch.empty(2, 16, device="cuda")
    mxq.moe_topk_backward(zc, ids, gw, dz)
    p = torch.softmax(zc.double().cpu(), 1)
    full = torch.zeros(2, 16, dtype=F64)
    full[0, 3] = 1.0
    within(dz, p * (full - (full * p).sum(1, keepdim=True)), 100 * HF)


# -------------------------------------------------------------------- sort

def sort_reference(ids, G):
    T, k = ids.shape
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < G))[0]
    order = kept[np.argsort(flat[kept], kind="stable")]
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=G)[:G])])
    pos = np.full(T * k, -1, np.int32)
    pos[order] = np.arange(order.size)
    src = np.full(T * k, -1, np.int32)
    src[:order.size] = order // k
    return off, src, pos.reshape(T, k)


def gpu_sort(ids, G, with_src=True):
    T, k = ids.shape
    off = torch.full((G + 1,), -9, dtype=torch.int64, device="cuda")
    src = torch.full((T * k,), -9, dtype=torch.int32, device="cuda") if with_src else None
    pos = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((max(16, mxq.moe_sort_workspace(T, k, G)),), 77, dtype=torch.uint8, device="cuda")
    mxq.moe_sort(torch.from_numpy(ids).cuda(), G, off, src, pos, ws)
    return off.cpu().numpy(), None if src is None else src.cpu().numpy(), pos.cpu().numpy()


@pytest.mark.parametrize("T,k,E,G", [(1, 1, 1, 1), (1, 8, 256, 32), (16, 8, 256, 256), (255, 8, 64, 64), (256, 8, 300, 300),
                                     (2011, 6, 100, 37), (16384, 10, 512, 512), (70001, 8, 600, 333), (3000, 4, 4096, 4096),
                                     (5000, 3, 5, 5)])
def test_sort(T, k, E, G):
    r = np.random.Generator(np.random.PCG64(T * k + G))
    ids = np.minimum((r.random((T, k)) ** 2 * E).astype(np.int32), E - 1)  # skewed
    off, src, pos = gpu_sort(ids, G)
    w_off, w_src, w_pos = sort_reference(ids, G)
    assert np.array_equal(off, w_off) and np.array_equal(pos, w_pos) and np.array_equal(src, w_src)


@pytest.mark.parametrize("T,k,E,G", [(131073, 8, 256, 256), (150001, 8, 9, 7), (16400, 8, 1030, 1024), (200000, 7, 1500, 1025),
                                     (1100, 4, 4096, 4095), (524300, 2, 300, 3)])
def test_sort_many_chunks(T, k, E, G):
    """More counts than every block should add up by itself."""
    r = np.random.Generator(np.random.PCG64(T + k + G))
    ids = r.integers(-1, E, (T, k), dtype=np.int32)
    ids[T // 3:T // 2] = G - 1  # a long run of one expert
    off, src, pos = gpu_sort(ids, G)
    w_off, w_src, w_pos = sort_reference(ids, G)
    assert np.array_equal(off, w_off) and np.array_equal(pos, w_pos) and np.array_equal(src, w_src)


@pytest.mark.parametrize("T", [0, 3, 4001])
def test_sort_nothing_local_one_expert_and_bad_ids(T):
    for ids in (np.full((T, 4), 50, np.int32), np.full((T, 4), 3, np.int32),
                np.resize(np.array([-1, 2 ** 31 - 1, -2 ** 31, 5, 9], np.int32), (T, 4))):
        for with_src in (True, False):
            off, src, pos = gpu_sort(ids, 10, with_src)
            w_off, w_src, w_pos = sort_reference(ids, 10)
            assert np.array_equal(off, w_off) and np.array_equal(pos, w_pos)
            assert src is None or np.array_equal(src, w_src)


# ---------------------------------------------------------------- movement

def routing(T, k, E, G, seed, capacity=None):
    """Distinct experts per token and the rows of the local ones; rows past the capacity are dropped."""
    r = np.random.Generator(np.random.PCG64(seed))
    ids = np.argsort(r.random((T, E)), axis=1)[:, :k].astype(np.int32)
    pos = sort_reference(ids, G)[2]
    n = int((pos >= 0).sum())
    return torch.from_numpy(pos), n if capacity is None else capacity


@pytest.mark.parametrize("fmt", [mxq.E4M3, mxq.E5M2, mxq.E2M1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,C,k,E,G", [(1, 32, 1, 4, 4), (3, 64, 2, 8, 3), (100, 96, 8, 16, 16), (37, 2080, 3, 16, 5),
                                       (64, 7168, 8, 64, 8)])
def test_dispatch_is_the_quantizer_then_the_copy(T, C, k, E, G, dtype, fmt):
    pos, R = routing(T, k, E, G, T + C)
    R = max(R, 1) + 2
    x = torch.randn(T, C + 16, generator=gen(C)) * 3
    x[:, 5] *= 1e4
    x[T // 2, :32] = 0.0
    x[T - 1, 1] = float("nan")
    x = x.to(dtype).cuda()[:, :C]  # a row pitch of its own
    cpb = C // 2 if fmt == mxq.E2M1 else C
    u8 = lambda *s: torch.full(s, 0xA5, dtype=torch.uint8, device="cuda")
    q, s, qx, sx = u8(R, cpb), u8(R, C // 32), u8(T, cpb), u8(T, C // 32)
    mxq.quantize_mx(x, fmt, qx, sx)
    mxq.moe_dispatch_mx(x, pos.cuda(), fmt, q, s)
    want_q, want_s = u8(R, cpb), u8(R, C // 32)
    for j in range(k):
        at = (pos[:, j] >= 0).nonzero()[:, 0].cuda()
        to = pos[:, j].cuda().long()[at]
        want_q[to], want_s[to] = qx[at], sx[at]
    assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_dispatch_every_exponent():
    """Blocks of every binary32 magnitude, subnormals and the largest included, as the quantizer casts them."""
    e = torch.arange(256, dtype=torch.int64)
    bits = (e[:, None] << 23) | (torch.arange(64, dtype=torch.int64)[None] * 0x1FFFF & 0x7FFFFF)
    bits[:, 1::2] |= 1 << 31
    bits[:, 32:] = torch.where(e[:, None] >= 6, bits[:, 32:] - (3 << 23), bits[:, 32:])
    x = (bits & 0xFFFFFFFF).to(torch.int64).numpy().astype(np.uint32).view(np.float32)
    x = torch.from_numpy(x.copy()).cuda()
    pos = torch.arange(256, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    for src in (x, x.to(BF)):
        for fmt in (mxq.E4M3, mxq.E5M2, mxq.E2M1):
            cpb = 32 if fmt == mxq.E2M1 else 64
            out = [torch.empty(256, n, dtype=torch.uint8, device="cuda") for n in (cpb, 2, cpb, 2)]
            mxq.quantize_mx(src, fmt, out[0], out[1])
            mxq.moe_dispatch_mx(src, pos, fmt, out[2], out[3])
            assert torch.equal(out[2], out[0].flip(0)) and torch.equal(out[3], out[1].flip(0))


def test_dispatch_entries_outside_the_buffers_are_left_out():
    x = torch.randn(3, 64, generator=gen(2)).to(BF).cuda()
    pos = torch.tensor([[0, 4], [-1, -2 ** 31], [2 ** 31 - 1, 3]], dtype=torch.int32, device="cuda")
    q, s = (torch.full((4, n), 1, dtype=torch.uint8, device="cuda") for n in (64, 2))
    qx, sx = (torch.empty(3, n, dtype=torch.uint8, device="cuda") for n in (64, 2))
    mxq.quantize_mx(x, mxq.E4M3, qx, sx)
    mxq.moe_dispatch_mx(x, pos, mxq.E4M3, q, s)
    assert torch.equal(q[0], qx[0]) and torch.equal(q[3], qx[2]) and bool((q[1:3] == 1).all())
    assert torch.equal(s[0], sx[0]) and torch.equal(s[3], sx[2]) and bool((s[1:3] == 1).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,C,k,E,G,weighted", [(1, 8, 1, 2, 2, True), (5, 24, 2, 8, 4, False), (16, 7168, 8, 64, 64, True),
                                                (33, 2056, 6, 16, 3, True), (7, 64, 70, 80, 80, True),
                                                (300, 520, 3, 9, 9, False)])
def test_combine_and_its_gradient(T, C, k, E, G, weighted, dtype):
    pos, R = routing(T, k, E, G, T * C, None)
    R = max(R - 1, 1)  # the last row is past the buffer: dropped
    g = gen(T + C)
    rows = torch.randn(R, C + 8, generator=g).to(dtype)
    w = torch.rand(T, k, generator=g)
    dy = torch.randn(T, C, generator=g).to(dtype)
    at = torch.where((pos < 0) | (pos >= R), R, pos).long()
    table = torch.cat([rows[:, :C].double(), torch.zeros(1, C, dtype=F64)])[at]  # [T, k, C]
    wd = (w if weighted else torch.ones_like(w)).double()
    want = (wd[..., None] * table).sum(1)
    size = (wd[..., None] * table).abs().sum(1)
    y = torch.full((T, C + 8), 5.0, dtype=dtype, device="cuda")
    mxq.moe_combine(rows.cuda()[:, :C], pos.cuda(), y[:, :C], weights=w.cuda() if weighted else None)
    within(y[:, :C], want, (k + 1) * HF * size + H[dtype] * want.abs() + TINY, "combine")
    assert bool((y[:, C:] == 5.0).all())
    if k > 64:
        return
    drows = torch.full((R, C + 8), 7.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), 7.0, device="cuda")
    mxq.moe_combine_backward(dy.cuda(), pos.cuda(), drows[:, :C], weights=w.cuda() if weighted else None,
                             rows=rows.cuda()[:, :C], dweights=dw)
    want_dw = (table * dy.double()[:, None]).sum(2)
    within(dw, want_dw, (C + 1) * HF * (table * dy.double()[:, None]).abs().sum(2) + TINY, "dweights")
    want_dx = torch.full((R + 1, C), 7.0, dtype=F64)
    want_dx[at.reshape(-1)] = (wd[..., None] * dy.double()[:, None]).reshape(-1, C)
    within(drows[:, :C], want_dx[:R], (HF + H[dtype]) * want_dx[:R].abs() + TINY, "drows")
    assert bool((drows[:, C:] == 7.0).all())
    only = torch.full((R, C), 7.0, dtype=dtype, device="cuda")
    mxq.moe_combine_backward(dy.cuda(), pos.cuda(), only, weights=w.cuda() if weighted else None)
    assert torch.equal(only, drows[:, :C])
    dw2 = torch.empty(T, k, device="cuda")
    mxq.moe_combine_backward(dy.cuda(), pos.cuda(), rows=rows.cuda()[:, :C], dweights=dw2)
    assert torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,C,k,E,G,weighted", [(1, 512, 64, 64, 64, True), (3, 1000, 63, 70, 64, True), (2, 2056, 64, 64, 60, False),
                                                (5, 4000, 9, 12, 12, True), (2, 9000, 33, 40, 40, True), (4101, 64, 5, 7, 6, True),
                                                (1026, 264, 3, 5, 5, False), (127, 7328, 8, 8, 7, True), (514, 1032, 1, 2, 1, True)])
def test_combine_gradient_rows_of_every_width(T, C, k, E, G, weighted, dtype):
    """A wave or a block per row, and the places of few tokens cut over blocks."""
    test_combine_and_its_gradient(T, C, k, E, G, weighted, dtype)


def test_combine_nothing_to_combine_and_non_finite_rows_elsewhere():
    rows = torch.full((4, 64), float("nan"), dtype=BF, device="cuda")
    rows[2] = 1.0
    pos = torch.tensor([[-1, -1], [2, -1], [4, 99]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan"), 1.0], [0.5, float("nan")], [1.0, 1.0]], device="cuda")
    y = torch.full((3, 64), 3.0, dtype=BF, device="cuda")
    mxq.moe_combine(rows, pos, y, weights=w)
    assert y.float().sum(1).tolist() == [0.0, 32.0, 0.0]
    dw = torch.full((3, 2), 3.0, device="cuda")
    mxq.moe_combine_backward(torch.ones(3, 64, dtype=BF, device="cuda"), pos, rows=rows, dweights=dw)
    assert dw.tolist() == [[0.0, 0.0], [64.0, 0.0], [0.0, 0.0]]
    empty = torch.empty(0, 64, dtype=BF, device="cuda")
    mxq.moe_combine(empty, pos, y)
    assert not bool(y.any())


# ----------------------------------------------------------- cross entropy

def lce_reference(x, w, t, dloss):
    """Definition in 64 bits on the CPU, with the sizes that its bounds take."""
    x, w = x.double(), w.double()
    T, V = x.shape[0], w.shape[0]
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    ok = (t >= 0) & (t < V)
    at = t.clamp(0, V - 1)[:, None]
    loss = torch.where(ok, lse - z.gather(1, at)[:, 0], 0.0)
    p = (z - lse[:, None]).exp()
    g = p.scatter_add(1, at, -torch.ones(T, 1, dtype=F64, device=x.device)) * torch.where(ok, dloss.double(), 0.0)[:, None]
    r = torch.where(ok, dloss.double(), 0.0)[:, None].abs()
    ez = (x.shape[1] + 1) * HF * (x.abs() @ w.abs().t())  # each logit
    return dict(z=z, lse=lse, loss=loss, g=g, p=p, r=r, ez=ez, ok=ok, dx=g @ w, dw=g.t() @ x, x=x, w=w)


def lce_bounds(ref, T, V, Hd):
    """lse: the largest logit's error, the fast exponentials of the tiles and of their join, a sum of V terms, the log.
    g: its rounding to bf16 (relative to the largest |dloss|: one binary32 quotient more), the exponential, the logit
    and lse.  dx, dw: g's errors, binary32 sums over V or T terms, the output's half step."""
    spread = (ref["z"] - ref["lse"][:, None]).abs().amax(1)
    e_exp = 4 * (2 + spread) * HF  # two exponentials, each with its argument's size
    e_lse = ref["ez"].amax(1) + e_exp + (V + 8) * HF + 4 * HF * ref["lse"].abs()
    e_loss = e_lse + ref["ez"].amax(1) + 2 * HF * (ref["lse"].abs() + ref["z"].abs().amax(1))
    e_g = (2.0 ** -8 + 8 * HF) * ref["g"].abs() + ref["p"] * ref["r"] * (ref["ez"] + e_lse[:, None] + e_exp[:, None])
    e_g = e_g + HF * ref["r"]  # 1 - p near 1
    e_g = e_g + TINY * ref["r"].max()  # what underflows
    g, x, w = ref["g"].abs() + e_g, ref["x"].abs(), ref["w"].abs()
    e_dx = e_g @ w + (V + 66) * HF * (g @ w) + 2.0 ** -8 * ref["dx"].abs() + TINY
    e_dw = e_g.t() @ x + (T + 2) * HF * (g.t() @ x) + 2.0 ** -8 * ref["dw"].abs() + TINY
    return e_lse, e_loss, 1.01 * e_dx, 1.01 * e_dw


def gpu_lce(x, w, t, dloss, want_dx=True, want_dw=True, pitch=0):
    T, Hd = x.shape
    V = w.shape[0]
    ws = torch.full((mxq.linear_cross_entropy_workspace(T, Hd, V, True),), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.full((T,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda")
    wide = lambda a: torch.full((a.shape[0], Hd + pitch), 7.0, dtype=BF, device="cuda")[:, :Hd]
    xd, wd = wide(x), wide(w)
    xd.copy_(x)
    wd.copy_(w)
    dx, dw = wide(x) if want_dx else None, wide(w) if want_dw else None
    mxq.linear_cross_entropy(xd, wd, t.cuda(), loss, lse, ws)
    ws.fill_(0xFF)  # nothing is kept from the forward call
    mxq.linear_cross_entropy_backward(xd, wd, t.cuda(), lse, dloss.cuda(), dx, dw, ws)
    return loss, lse, dx, dw


def lce_case(T, Hd, V, seed, ignored=0.2, std=1.5):
    g = gen(seed)
    x = torch.randn(T, Hd, generator=g).to(BF)
    w = (torch.randn(V, Hd, generator=g) * std / Hd ** 0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -100
    dloss = torch.randn(T, generator=g)
    return x, w, t, dloss


@pytest.mark.parametrize("T,Hd,V,pitch", [(1, 8, 1, 0), (1, 64, 300, 8), (3, 72, 7, 0), (48, 128, 1000, 0), (64, 64, 129, 24),
                                          (65, 136, 515, 0), (128, 256, 2049, 0), (129, 64, 256, 0), (200, 200, 777, 40),
                                          (256, 512, 1024, 0), (257, 328, 3001, 0), (600, 72, 65, 8), (1031, 264, 700, 0),
                                          (10, 4000, 500, 0), (33, 2056, 901, 0), (20, 1032, 3000, 16), (1, 520, 40, 0)])
def test_cross_entropy(T, Hd, V, pitch):
    x, w, t, dloss = lce_case(T, Hd, V, T + V)
    ref = lce_reference(x, w, t, dloss)
    e_lse, e_loss, e_dx, e_dw = lce_bounds(ref, T, V, Hd)
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss, pitch=pitch)
    within(lse, ref["lse"], e_lse, "lse")
    within(loss, ref["loss"], torch.where(ref["ok"], e_loss, 0.0), "loss")
    within(dx, ref["dx"], e_dx, "dx")
    within(dw, ref["dw"], e_dw, "dw")
    if pitch:
        for a in (dx, dw):
            assert bool((a.as_strided((a.shape[0], pitch), (Hd + pitch, 1), Hd) == 7.0).all())
    one = gpu_lce(x, w, t, dloss, want_dw=False)
    two = gpu_lce(x, w, t, dloss, want_dx=False)
    assert torch.equal(one[2], dx) and torch.equal(two[3], dw)  # the same from run to run


@pytest.mark.parametrize("T,Hd,V", [(2050, 512, 7717), (1025, 1024, 16001), (1100, 576, 30011), (2011, 2880, 9000)])
def test_cross_entropy_on_large_tiles(T, Hd, V):
    """More than a round of the large tiles, whose last words go to smaller ones."""
    _on_the_gpu(T, Hd, V)


def test_cross_entropy_in_several_pieces():
    """Enough tokens that the vocabulary is cut into pieces, at an odd end."""
    _on_the_gpu(40000, 16, 4133)


def _on_the_gpu(T, Hd, V):
    """Against the definition in 64 bits on the GPU."""
    x, w, t, dloss = lce_case(T, Hd, V, 3)
    dev = [a.cuda() for a in (x, w, t, dloss)]
    ref = lce_reference(*dev)
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss)
    e_lse, e_loss, e_dx, e_dw = lce_bounds(ref, T, V, Hd)
    for got, want, bound, what in ((lse, ref["lse"], e_lse, "lse"), (dx, ref["dx"], e_dx, "dx"),
                                   (dw, ref["dw"], e_dw, "dw")):
        within(got, want.cpu(), bound.cpu(), what)


def test_cross_entropy_in_two_equal_pieces():
    """g of the whole vocabulary would be more than twice what a piece may take."""
    _on_the_gpu(70000, 16, 8133)


@pytest.mark.parametrize("T,Hd,V", [(5, 520, 105001), (66, 1032, 130007), (127, 512, 31999), (100, 5120, 9001), (300, 264, 40001)])
def test_cross_entropy_of_few_tokens_and_many_words(T, Hd, V):
    """Where w's gradient is bound by its stores, or a product has one block per CU."""
    _on_the_gpu(T, Hd, V)


@pytest.mark.parametrize("T,Hd,V", [(1, 264, 44001), (64, 1032, 15001), (129, 1000, 17001), (256, 1024, 16385)])
def test_cross_entropy_gradient_of_the_projection_alone(T, Hd, V):
    x, w, t, dloss = lce_case(T, Hd, V, 4)
    ref = lce_reference(*[a.cuda() for a in (x, w, t, dloss)])
    _, lse, dx, dw = gpu_lce(x, w, t, dloss, want_dx=False)
    e_lse, _, _, e_dw = lce_bounds(ref, T, V, Hd)
    assert dx is None
    within(lse, ref["lse"].cpu(), e_lse.cpu(), "lse")
    within(dw, ref["dw"].cpu(), e_dw.cpu(), "dw")


@pytest.mark.parametrize("T", [3, 300])
def test_cross_entropy_ignored_tokens_and_targets_out_of_range(T):
    x, w, t, dloss = lce_case(T, 64, 500, 8, ignored=0.0)
    t[0], t[1], t[2] = 500, 2 ** 40, -2 ** 63
    dloss[:3] = float("nan")  # of tokens that do not count
    ref = lce_reference(x, w, t, dloss)
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss)
    e_lse, e_loss, e_dx, e_dw = lce_bounds(ref, T, 500, 64)
    assert loss[:3].tolist() == [0.0] * 3 and not bool(dx[:3].any())
    within(loss, ref["loss"], e_loss, "loss")
    within(dx, ref["dx"], e_dx, "dx")
    within(dw, ref["dw"], e_dw, "dw")
    none = gpu_lce(x, w, torch.full((T,), -100), dloss)
    assert not bool(none[0].any()) and not bool(none[2].any()) and not bool(none[3].any())
    zero = gpu_lce(x, w, t, torch.zeros(T))
    assert not bool(zero[2].any()) and not bool(zero[3].any())


@pytest.mark.parametrize("T", [2, 200])
def test_cross_entropy_large_and_confident_logits(T):
    """Logits of a few hundred: exp overflows without the maximum; all of them far below zero; a probability of one."""
    x, w, t, dloss = lce_case(T, 64, 300, 9, ignored=0.0, std=60.0)
    x[1] = 4.0
    t[0] = int((x[0].double() @ w.double().t()).argmax())
    ref = lce_reference(x, w, t, dloss)
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss)
    e_lse, e_loss, e_dx, e_dw = lce_bounds(ref, T, 300, 64)
    for a, b, e, n in ((lse, "lse", e_lse, "lse"), (loss, "loss", e_loss, "loss"), (dx, "dx", e_dx, "dx"),
                       (dw, "dw", e_dw, "dw")):
        within(a, ref[b], e, n)
    x = torch.full((T, 64), 2.0).to(BF)
    w = torch.full((300, 64), -3.0).to(BF)  # every logit -384: a tile's unused rows must not raise the maximum
    loss, lse, _, _ = gpu_lce(x, w, t, dloss)
    within(lse, torch.full((T,), -384.0 + np.log(300.0), dtype=F64), 1e-4)


def test_cross_entropy_nan_and_infinity_reach_their_own_token():
    x, w, t, dloss = lce_case(300, 64, 400, 10, ignored=0.0)
    x[7, 3], x[9, 5] = float("nan"), float("inf")
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss)
    bad = torch.zeros(300, dtype=torch.bool)
    bad[7] = bad[9] = True
    assert torch.equal(loss.isnan().cpu() | loss.isinf().cpu(), bad)
    assert torch.equal(dx.isnan().any(1).cpu(), bad)


def test_cross_entropy_no_tokens():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(37, 64, dtype=BF, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    f = lambda: torch.empty(0, device="cuda")
    ws = torch.empty(mxq.linear_cross_entropy_workspace(0, 64, 37, True), dtype=torch.uint8, device="cuda")
    mxq.linear_cross_entropy(x, w, t, f(), f(), ws)
    dw = torch.ones_like(w)
    mxq.linear_cross_entropy_backward(x, w, t, f(), f(), torch.empty_like(x), dw, ws)
    assert not bool(dw.any())


def test_cross_entropy_gradient_against_differences():
    """The kernel's gradients along a direction against central differences of the loss in 64 bits."""
    T, Hd, V = 150, 64, 401
    x, w, t, dloss = lce_case(T, Hd, V, 12)
    loss, lse, dx, dw = gpu_lce(x, w, t, dloss)
    g = gen(13)
    ux, uw = torch.randn(T, Hd, generator=g).double(), torch.randn(V, Hd, generator=g).double()
    f = lambda h, a, b: float((lce_reference(x.double() + h * a, w.double() + h * b, t, dloss)["loss"] * dloss.double()).sum())
    ref = lce_reference(x, w, t, dloss)
    _, _, e_dx, e_dw = lce_bounds(ref, T, V, Hd)
    for got, u, bound, slope in ((dx, ux, e_dx, lambda h: f(h, ux, 0 * uw) - f(-h, ux, 0 * uw)),
                                 (dw, uw, e_dw, lambda h: f(h, 0 * ux, uw) - f(-h, 0 * ux, uw))):
        h = 1e-5
        want = slope(h) / (2 * h)
        assert abs(float((got.cpu().double() * u).sum()) - want) <= float((bound * u.abs()).sum()) + 1e-5 * abs(want) + 1e-4


# ---------------------------------------------------------------- clipping

@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0])
@pytest.mark.parametrize("where", ["in place", "apart", "misaligned"])
def test_clip(max_norm, where):
    g = gen(21)
    sizes = [1, 7, 0, 16384, 16385, 40000, 3, 8, 2049, 131072]
    host, grads, out = [], [], []
    for n, size in enumerate(sizes):
        dt = BF if n % 3 else F32
        h = torch.randn(size + 3, generator=g).to(dt)
        d = h.cuda()
        a = 0 if where != "misaligned" else n % 4
        host.append(h[a:a + size])
        grads.append(d[a:a + size])
        out.append(grads[-1] if where == "in place" else
                   torch.full((size + 3,), 3.0, dtype=dt, device="cuda")[0 if where == "apart" else 1:][:size])
    norm = torch.zeros(1, device="cuda")
    s = mxq.GradientSet(grads, None if where == "in place" else out)
    s.clip(max_norm, norm)
    want = float(torch.cat([h.double() for h in host]).square().sum().sqrt())
    within(norm, torch.tensor([want], dtype=F64), 2 * HF * want)
    coef = min(1.0, max_norm / (want + 1e-6))
    for h, o in zip(host, out):
        ref = h.double() * coef
        within(o, ref, (4 * HF + H[h.dtype]) * ref.abs() + TINY)


@pytest.mark.parametrize("big", [1025 * 8192 - 3, 4000 * 8192 + 1, 4100 * 8192])
def test_clip_many_chunks(big):
    """More chunks than partial sums, and more than the blocks add up themselves."""
    g = gen(22)
    host = [torch.randn(n, generator=g).to(dt) for n, dt in ((big, BF), (5, F32), (20000, F32))]
    grads, out = [h.cuda() for h in host], [torch.empty_like(h, device="cuda") for h in host]
    norm = torch.zeros(1, device="cuda")
    mxq.GradientSet(grads, out).clip(1.0, norm)
    want = float(sum(h.double().square().sum() for h in host).sqrt())
    within(norm, torch.tensor([want], dtype=F64), 2 * HF * want)
    for h, o in zip(host, out):
        ref = h.double() / (want + 1e-6)
        within(o, ref, (4 * HF + H[h.dtype]) * ref.abs() + TINY)


def test_clip_extreme_and_non_finite_values():
    for v, want in ((1e30, 1e30), (1e-30, 1e-30), (float("inf"), float("inf")), (float("nan"), float("nan"))):
        a, b = torch.zeros(100, device="cuda"), torch.ones(5, dtype=BF, device="cuda") * 0
        a[3] = v
        norm = torch.empty(1, device="cuda")
        mxq.GradientSet([a, b]).clip(1.0, norm)
        within(norm, torch.tensor([want], dtype=F64), 2 * HF * abs(want))
        if want == 1e30:
            assert abs(float(a[3]) - 1.0) < 1e-6
        if want == 1e-30:
            assert float(a[3]) == np.float32(1e-30)
        if want != want:
            assert bool(a.isnan().all()) and bool(b.isnan().all())
    one = torch.full((7,), 3.0, device="cuda")
    one[0] = float("inf")
    mxq.GradientSet([one]).clip(1.0, norm)
    assert bool(one[0].isnan()) and not bool(one[1:].any())  # inf * 0, 3 * 0


# ------------------------------------------------- streams, graphs, addresses

def test_a_gradient_set_let_go_while_another_stream_uses_it():
    """Its tables are not handed out again before the clipping that reads them is done."""
    a, norm = torch.full((1000,), 2.0, device="cuda"), torch.zeros(1, device="cuda")
    s = mxq.GradientSet([a])
    place, bytes_ = s._tables.data_ptr(), s._tables.nbytes
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        s.clip(1.0, norm)
    del s
    held = [torch.empty(bytes_, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert place not in [h.data_ptr() for h in held]
    torch.cuda.synchronize()
    want = float(np.sqrt(4000.0))
    within(norm, torch.tensor([want], dtype=F64), 2 * HF * want)
    within(a, torch.full((1000,), 2.0, dtype=F64) / (want + 1e-6), 8 * HF * torch.ones(1000, dtype=F64))


def test_a_step_on_another_stream_and_in_a_graph():
    """Router, sort, dispatch, combine, loss and clipping in one captured graph, replayed on new inputs between eager
    work, and on a stream of their own: each replay equals the eager calls."""
    T, E, k, C, V = 130, 16, 4, 128, 1000
    g = gen(31)
    z, x = torch.randn(T, E, generator=g).cuda(), torch.randn(T, C, generator=g).to(BF).cuda()
    w = (torch.randn(V, C, generator=g) * 0.1).to(BF).cuda()
    t = torch.randint(0, V, (T,), generator=g).cuda()
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")
    ids, wt, off, src, pos = i32(T, k), f(T, k), torch.empty(E + 1, dtype=torch.int64, device="cuda"), i32(T * k), i32(T, k)
    ws = torch.empty(max(16, mxq.moe_sort_workspace(T, k, E)), dtype=torch.uint8, device="cuda")
    q, s = (torch.empty(T * k, n, dtype=torch.uint8, device="cuda") for n in (C, C // 32))
    rows, y = torch.empty(T * k, C, dtype=BF, device="cuda"), torch.empty(T, C, dtype=BF, device="cuda")
    loss, lse, dl = f(T), f(T), torch.full((T,), 1.0 / T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    lws = torch.empty(mxq.linear_cross_entropy_workspace(T, C, V, True), dtype=torch.uint8, device="cuda")
    drows, dwt, dz, norm = torch.empty_like(rows), f(T, k), torch.empty_like(z), f(1)
    clipped = [torch.empty_like(a) for a in (dx, dw, dz)]
    grads = mxq.GradientSet([dx, dw, dz], clipped)

    def step():
        mxq.moe_topk(z, ids, wt, renormalize=True)
        mxq.moe_sort(ids, E, off, src, pos, ws)
        mxq.moe_dispatch_mx(x, pos, mxq.E4M3, q, s)
        rows.copy_(q.view(torch.float8_e4m3fn).to(BF))
        mxq.moe_combine(rows, pos, y, weights=wt)
        mxq.linear_cross_entropy(y, w, t, loss, lse, lws)
        mxq.linear_cross_entropy_backward(y, w, t, lse, dl, dx, dw, lws)
        mxq.moe_combine_backward(dx, pos, drows, weights=wt, rows=rows, dweights=dwt)
        mxq.moe_topk_backward(z, ids, dwt, dz, renormalize=True)
        grads.clip(1e-3, norm)

    outs = [ids, wt, off, src, pos, q, s, y, loss, lse, dx, dw, drows, dwt, dz, norm, *clipped]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(4):
        z.copy_(torch.randn(T, E, generator=g))
        x.copy_(torch.randn(T, C, generator=g))
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Row buffers of more than 4 GiB: the last rows are the ones that move."""
    C, R = 8192, 300_000  # bf16: 4.9 GB
    rows = torch.empty(R, C, dtype=BF, device="cuda")
    rows[R - 2:] = torch.arange(2, device="cuda")[:, None] + 1
    pos = torch.tensor([[R - 1, R - 2], [R - 2, -1]], dtype=torch.int32, device="cuda")
    y = torch.empty(2, C, dtype=BF, device="cuda")
    mxq.moe_combine(rows, pos, y)
    assert bool((y[0] == 3).all()) and bool((y[1] == 1).all())
    pos = torch.tensor([[R - 1], [R - 2]], dtype=torch.int32, device="cuda")
    mxq.moe_combine_backward(y, pos, rows)
    assert bool((rows[R - 1] == 3).all()) and bool((rows[R - 2] == 1).all())
    q, s = torch.zeros(R * 2, C, dtype=torch.uint8, device="cuda"), torch.zeros(R * 2, C // 32, dtype=torch.uint8, device="cuda")
    mxq.moe_dispatch_mx(y, pos + R, mxq.E4M3, q, s)
    assert bool((q[2 * R - 1] != 0).all()) and bool((q[2 * R - 2] != 0).all()) and not bool(q[2 * R - 3].any())


def test_cross_entropy_projection_past_32_bits():
    """A projection of 4.9 GB: its last words' logits and gradients, which lie past 2^32 bytes."""
    T, Hd, V, last = 16, 8192, 300_000, 128
    x, _, _, dloss = lce_case(T, Hd, 8, 40)
    w = torch.zeros(V, Hd, dtype=BF, device="cuda")  # every other logit is 0
    tail = (torch.randn(last, Hd, generator=gen(41)) * 2 / Hd ** 0.5).to(BF)
    w[V - last:] = tail.cuda()
    t = V - 1 - torch.arange(T)
    ws = torch.empty(mxq.linear_cross_entropy_workspace(T, Hd, V, True), dtype=torch.uint8, device="cuda")
    loss, lse, xd, dx, dw = (torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), x.cuda(), x.cuda(), w.clone())
    mxq.linear_cross_entropy(xd, w, t.cuda(), loss, lse, ws)
    mxq.linear_cross_entropy_backward(xd, w, t.cuda(), lse, dloss.cuda(), dx, dw, ws)
    z = x.double() @ tail.double().t()
    want = torch.log((V - last) + z.exp().sum(1))
    g = ((z - want[:, None]).exp() - torch.nn.functional.one_hot(t - (V - last), last)) * dloss.double()[:, None]
    ez = (Hd + 1) * HF * (x.double().abs() @ tail.double().abs().t()).amax(1)
    e_lse = ez + (V + 8) * HF + 8 * (2 + want) * HF
    within(lse, want, e_lse, "lse")
    within(loss, want - z.gather(1, (t - (V - last))[:, None])[:, 0], 2 * e_lse + ez, "loss")
    # g: bf16, the exponential and its argument; then binary32 sums and the output's half step
    e_g = 2.0 ** -8 * 1.01 * g.abs() + (ez + e_lse)[:, None] * (z - want[:, None]).exp() * dloss.double().abs()[:, None] + \
        2 * HF * dloss.double().abs()[:, None]
    e_dx = e_g @ tail.double().abs() + (V + 66) * HF * (g.abs() @ tail.double().abs())
    within(dx, g @ tail.double(), 1.01 * e_dx + 2.0 ** -8 * (g @ tail.double()).abs(), "dx")
    want_dw = g.t() @ x.double()
    e_dw = e_g.t() @ x.double().abs() + (T + 2) * HF * (g.abs().t() @ x.double().abs())
    within(dw[V - last:], want_dw, 1.01 * e_dw + 2.0 ** -8 * want_dw.abs(), "dw")
    p0 = ((-want).exp() * dloss.double()) @ x.double()  # the words whose logits are 0
    within(dw[V - last - 1], p0, 2.0 ** -7 * (((-want).exp() * dloss.double().abs()) @ x.double().abs()), "dw before")
