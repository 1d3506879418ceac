"""GPU tests of the training-step operators with more rows than one launch has
threads for (2^32): every row is computed, the first, the last and those at a
launch's end like the others.  Tolerances as in test_gpu_train_ops.py."""
import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from gpu_helpers import require_gpu
from test_gpu_train_ops import BF, F64, H, HF, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def needs(gib):
    free = torch.cuda.mem_get_info()[0] >> 30
    if free < gib:
        pytest.skip(f"{free} GiB free of the {gib} that the case takes")


def dgen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, bound, what):
    worst = float(((got.double() - want).abs() - bound).max())
    assert worst <= 0, f"{what}: beyond the bound by {worst:.3g}"  # a NaN too


def test_router_and_its_gradient():
    T = (1 << 26) + 5
    z = torch.randn(T, 2, generator=dgen(1), device="cuda", dtype=BF)
    ids, w = torch.full((T, 1), -7, dtype=torch.int32, device="cuda"), torch.full((T, 1), -7.0, device="cuda")
    mxq.moe_topk(z, ids, w)
    assert torch.equal(ids[:, 0] == 1, z[:, 1] > z[:, 0]) and int(ids.min()) == 0 and int(ids.max()) == 1
    d = (z[:, 0].double() - z[:, 1].double()).abs()
    p = 1 / (1 + (-d).exp())
    near(w[:, 0], p, (10 + 2 * d) * HF * p, "weights")
    g = torch.randn(T, 1, generator=dgen(2), device="cuda")
    dz = torch.full((T, 2), 9.0, dtype=BF, device="cuda")
    mxq.moe_topk_backward(z, ids, g, dz)
    want = p * (1 - p) * g[:, 0].double()  # of the chosen one; minus that of the other
    bound = (68 * HF) * p * 2 * g[:, 0].abs().double() + H[BF] * want.abs() + TINY
    near(dz.gather(1, ids.long())[:, 0], want, bound, "chosen")
    near(dz.gather(1, 1 - ids.long())[:, 0], -want, bound, "the other")


def test_gradient_of_the_combining_weights():
    T, C = (1 << 24) + 3, 1032
    needs(40)
    at = torch.cat([torch.arange(3), (1 << 23) + torch.arange(-3, 3), T - 1 - torch.arange(5)]).cuda()
    dy = torch.zeros(T, C, dtype=BF, device="cuda")
    dy[at] = torch.randn(at.numel(), C, generator=dgen(3), device="cuda").to(BF)
    rows = torch.randn(4, C, generator=dgen(4), device="cuda").to(BF)
    pos = torch.randint(0, 4, (T, 1), generator=dgen(5), device="cuda", dtype=torch.int32)
    dw = torch.full((T, 1), 7.0, device="cuda")
    mxq.moe_combine_backward(dy, pos, rows=rows, dweights=dw)
    terms = rows[pos[at, 0].long()].double() * dy[at].double()
    near(dw[at, 0], terms.sum(1), (C + 1) * HF * terms.abs().sum(1) + TINY, "dweights")
    dw[at] = 0.0
    assert not bool(dw.any())


def lse_of(x, w, t):
    """z, lse and loss in 64 bits, and the bound of each logit's sum."""
    x, w = x.double(), w.double()
    z = (x[:, None] * w[None]).sum(2) if w.shape[0] < 64 else torch.mm(x, w.t().contiguous())
    ez = (x.shape[1] + 1) * HF * torch.mm(x.abs(), w.abs().t().contiguous()).amax(1)
    lse = torch.logsumexp(z, 1)
    return z, lse, lse - z.gather(1, t[:, None])[:, 0], ez


def check_loss(x, w, t, loss, lse):
    V = w.shape[0]
    z, want_lse, want, ez = lse_of(x, w, t)
    spread = (z - want_lse[:, None]).abs().amax(1)
    e_lse = ez + 4 * (2 + spread) * HF + (V + 8) * HF + 4 * HF * want_lse.abs()
    near(lse, want_lse, e_lse, "lse")
    near(loss, want, e_lse + ez + 2 * HF * (want_lse.abs() + z.abs().amax(1)), "loss")


def test_statistics_of_many_tokens():
    T, Hd, V = (1 << 25) + 9, 8, 5
    needs(20)
    x = torch.randn(T, Hd, generator=dgen(6), device="cuda", dtype=BF)
    w = torch.randn(V, Hd, generator=dgen(7), device="cuda", dtype=BF)
    t = torch.randint(0, V, (T,), generator=dgen(8), device="cuda")
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    ws = torch.empty(mxq.linear_cross_entropy_workspace(T, Hd, V), dtype=torch.uint8, device="cuda")
    mxq.linear_cross_entropy(x, w, t, loss, lse, ws)
    for a in range(0, T, 1 << 22):
        s = slice(a, a + (1 << 22))
        check_loss(x[s], w, t[s], loss[s], lse[s])


def test_tiles_of_many_tokens_and_words():
    T, Hd, V = (1 << 22) + 300, 8, 1 << 17
    needs(40)
    x = torch.randn(T, Hd, generator=dgen(9), device="cuda", dtype=BF)
    w = torch.randn(V, Hd, generator=dgen(10), device="cuda", dtype=BF)
    t = torch.randint(0, V, (T,), generator=dgen(11), device="cuda")
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.empty(mxq.linear_cross_entropy_workspace(T, Hd, V), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # statistics that no tile wrote would be NaN
    mxq.linear_cross_entropy(x, w, t, loss, lse, ws)
    assert bool(loss.isfinite().all()) and bool(lse.isfinite().all())
    at = torch.cat([torch.arange(64), torch.arange(0, T, T // 400), T - 1 - torch.arange(400)]).cuda()
    check_loss(x[at], w, t[at], loss[at], lse[at])


def test_gradients_of_many_tokens():
    T, Hd, V = (1 << 25) + 9, 512, 5
    needs(190)
    at = torch.cat([torch.arange(3), (1 << 24) + torch.arange(-3, 3), (1 << 25) + torch.arange(-3, 9)]).cuda()
    n = at.numel()
    x = torch.zeros(T, Hd, dtype=BF, device="cuda")
    x[at] = torch.randn(n, Hd, generator=dgen(12), device="cuda").to(BF)
    w = (torch.randn(V, Hd, generator=dgen(13), device="cuda") / Hd ** 0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=dgen(14), device="cuda")
    dloss = torch.zeros(T, device="cuda")
    dloss[at] = torch.randn(n, generator=dgen(15), device="cuda")
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    dx, dw = torch.full_like(x, 7.0), torch.empty_like(w)
    ws = torch.empty(mxq.linear_cross_entropy_workspace(T, Hd, V, True), dtype=torch.uint8, device="cuda")
    mxq.linear_cross_entropy(x, w, t, loss, lse, ws)
    mxq.linear_cross_entropy_backward(x, w, t, lse, dloss, dx, dw, ws)
    z, want_lse, _, ez = lse_of(x[at], w, t[at])
    p = (z - want_lse[:, None]).exp()
    r = dloss[at].double()[:, None]
    g = (p - torch.nn.functional.one_hot(t[at], V)) * r
    # g: bf16 (and the quotient by the largest |dloss|), the logit's and lse's errors; sums and the output's half step
    e_g = (2.0 ** -8 + 8 * HF) * g.abs() + p * r.abs() * (2 * ez + (V + 8) * HF + 20 * (2 + want_lse.abs()) * HF)[:, None]
    e_g = e_g + 2 * HF * r.abs()
    wa, xa = w.double().abs(), x[at].double().abs()
    want = torch.mm(g, w.double())
    near(dx[at], want, 1.01 * (torch.mm(e_g, wa) + 70 * HF * torch.mm(g.abs() + e_g, wa)) + H[BF] * want.abs(), "dx")
    dx[at] = 0.0
    assert not bool(dx.any())
    want = torch.mm(g.t().contiguous(), x[at].double())
    e_dw = torch.mm(e_g.t().contiguous(), xa) + (n + 2) * HF * torch.mm((g.abs() + e_g).t().contiguous(), xa)
    near(dw, want, 1.01 * e_dw + H[BF] * want.abs() + TINY, "dw")


def test_more_chunks_than_a_launch_has_threads_for():
    """2^24 + 3 chunks, of as many tensors of one element."""
    n = (1 << 24) + 3
    F = mxq.GradientSet
    data = torch.full((n,), 2.0, device="cuda")
    out = torch.zeros(n, device="cuda")
    i = torch.arange(n, device="cuda")
    tables = torch.stack([data.data_ptr() + 4 * i, out.data_ptr() + 4 * i, torch.ones_like(i), torch.full_like(i, mxq.SRC_F32),
                          i], 1).contiguous()  # in, out, numel, src and pad, first
    parts, norm = torch.empty(F.PARTS, dtype=F64, device="cuda"), torch.empty(1, device="cuda")
    from mxfp4_precision_numerics_amd import training
    of = i.to(torch.int32)
    status = training._lib().mxq_clip_grad_norm(tables.data_ptr(), n, of.data_ptr(), n, 1.0, norm.data_ptr(),
                                                parts.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    want = (4.0 * n) ** 0.5
    assert abs(float(norm) - want) <= 2 * HF * want
    near(out, torch.full((n,), 2.0 / (want + 1e-6), dtype=F64, device="cuda"), 4 * HF * 2.0 / want, "clipped")
