"""Linear and gated layers as a program calls them (GPU): pitched views and what lies beside them, outputs in place of
inputs, no tokens, values that are not finite, captured and replayed calls, other streams, shared workspaces, matrices beyond
2^32 elements, gradients one by one and against differences, and all of it together with the update.

Tolerances: those of test_gpu_dense_layers, and what the tests say.
"""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from test_gpu_dense_layers import ACTS, BF, DEV, F32, F64, HALF, SUM, act, bytes_, gradients, mm, near, rn, slope, sums

pytestmark = pytest.mark.gpu
NONE, SILU, GELU = mxq.ACT_NONE, mxq.ACT_SILU, mxq.ACT_GELU

# tokens, hidden, features (a gated layer's inter: half): rows, quick and wide tiles, splits, small and large tiles
SIZES = [(1, 264, 1008), (3, 2056, 48), (20, 520, 2000), (50, 1032, 1008), (24, 4096, 8208), (100, 2880, 24592), (300, 4096, 528),
         (700, 264, 4112), (1100, 520, 6016)]


class Wide:
    """A matrix inside a larger one whose other elements are known."""

    def __init__(self, rows, cols, dtype=BF, value=None):
        self.all = torch.full((rows + 5, cols + 24), 77.0, dtype=dtype, device=DEV)
        self.t = self.all[2:rows + 2, 8:cols + 8]
        if value is not None:
            self.t.copy_(value)

    def untouched(self):
        r, c = self.t.shape
        rest = self.all.clone()
        rest[2:r + 2, 8:c + 8] = 77.0
        return bool((rest == 77.0).all())


def calls(T, H, N, name, seed, make=None):
    """Every output of the forward and backward calls of both layers, each into matrices that `make` makes."""
    make = make or (lambda r, c, dtype=BF, value=None: torch.zeros(r, c, dtype=dtype, device=DEV) if value is None else value)
    I, out = N // 2, {}
    x, w, dy, r = rn(T, H, seed=seed), rn(N, H, seed=seed + 1, std=1 / math.sqrt(H)), rn(T, N, seed=seed + 2), rn(T, N, seed=seed + 3)
    dh, add, old = dy[:, :I].contiguous(), rn(T, H, seed=seed + 4), rn(N, H, seed=seed + 5, dtype=F32)
    b = rn(N, seed=seed + 6, dtype=F32)
    x, w, dy, r, dh, add = (make(*t.shape, value=t) for t in (x, w, dy, r, dh, add))
    y, z, h, gz = make(T, N), make(T, N), make(T, I), make(T, N)
    dx, dw, gdx, gdw = make(T, H), make(N, H, F32, old), make(T, H), make(N, H)
    db = torch.empty(N, device=DEV)
    ws = bytes_(max(f(T, H, n, k) for f, n in ((mxq.linear_workspace, N), (mxq.gated_linear_workspace, I)) for k in (0, 1)))
    at = lambda m: m.t if isinstance(m, Wide) else m
    mxq.linear(at(x), at(w), at(y), b, ACTS[name], at(r), at(z), ws)
    mxq.gated_linear(at(x), at(w), at(h), ACTS[name], at(gz), ws)
    mxq.linear_backward(at(x), at(w), at(dy), at(dx), at(dw), db, ACTS[name], at(z), at(add), False, ws)
    mxq.gated_linear_backward(at(x), at(w), at(dh), at(gdx), at(gdw), ACTS[name], at(gz), None, False, ws)
    out = dict(y=y, z=z, h=h, gz=gz, dx=dx, dw=dw, gdx=gdx, gdw=gdw, x=x, w=w, dy=dy, r=r, dh=dh, add=add)
    return {k: at(v).clone() for k, v in out.items()}, db, list(out.values())


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_pitched_views_and_what_lies_beside_them(n):
    T, H, N = SIZES[n]
    name = list(ACTS)[1 + n % 4]
    dense, db, _ = calls(T, H, N, name, 7 * n)
    pitched, db2, wide = calls(T, H, N, name, 7 * n, Wide)
    for k in dense:
        assert torch.equal(dense[k], pitched[k]), k
    assert torch.equal(db, db2)
    assert all(m.untouched() for m in wide)


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_in_place_of_an_input(n):
    """The residual may be y, add may be dx: bit for bit the result from elsewhere."""
    T, H, N = SIZES[n]
    x, w, dy = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H)), rn(T, N, seed=3)
    ws = bytes_(max(mxq.linear_workspace(T, H, N), mxq.linear_workspace(T, H, N, True)))
    for dtype in (BF, F32):
        r = rn(T, N, seed=4, dtype=dtype)
        y = torch.empty_like(r)
        mxq.linear(x, w, y, activation=GELU, residual=r, workspace=ws)
        mxq.linear(x, w, r, activation=GELU, residual=r, workspace=ws)
        assert torch.equal(y, r)
    z, add = rn(T, N, seed=5), rn(T, H, seed=6)
    dx = torch.empty_like(add)
    for more in ({}, dict(dw=torch.empty_like(w))):
        a = add.clone()
        mxq.linear_backward(x, w, dy, dx, activation=SILU, z=z, add=a, workspace=ws, **more)
        mxq.linear_backward(x, w, dy, a, activation=SILU, z=z, add=a, workspace=ws, **more)
        assert torch.equal(dx, a)


def test_no_tokens():
    H, N = 64, 48
    e, w = torch.empty(0, H, dtype=BF, device=DEV), rn(N, H, seed=1)
    y = torch.empty(0, N, dtype=BF, device=DEV)
    mxq.linear(e, w, y)
    mxq.gated_linear(e, w, y[:, :N // 2])
    for dtype in (BF, F32):
        for add in (True, False):
            dw, db = rn(N, H, seed=2, dtype=dtype), rn(N, seed=3, dtype=F32)
            want = (dw.clone(), db.clone()) if add else (torch.zeros_like(dw), torch.zeros_like(db))
            mxq.linear_backward(e, w, y, e, dw, db, GELU, y, accumulate=add)
            assert torch.equal(dw, want[0]) and torch.equal(db, want[1])
            dw = Wide(N, H, dtype, rn(N, H, seed=2, dtype=dtype))
            mxq.gated_linear_backward(e, w, y[:, :N // 2], e, dw.t, accumulate=add)
            assert torch.equal(dw.t, want[0]) and dw.untouched()


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_what_is_not_finite_stays_in_its_rows_and_columns(n):
    T, H, N = SIZES[n]
    x, w, dy = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H)), rn(T, N, seed=3)
    clean, _, _ = calls(T, H, N, "silu", 0)
    ws = bytes_(max(f(T, H, n, k) for f, n in ((mxq.linear_workspace, N), (mxq.gated_linear_workspace, N // 2)) for k in (0, 1)))
    y, h, z = torch.empty(T, N, dtype=BF, device=DEV), torch.empty(T, N // 2, dtype=BF, device=DEV), rn(T, N, seed=4)

    def only(a, b, rows, cols, what):
        """a is b but for some rows and columns, all of which are NaN or infinite."""
        hit = torch.zeros(a.shape, dtype=torch.bool, device=DEV)
        hit[rows], hit[:, cols] = True, True
        assert torch.equal(a[~hit], b[~hit]), what
        assert not bool(torch.isfinite(a[hit]).any()), what

    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    t, f = torch.tensor([T // 2], device=DEV), torch.tensor([N // 2 - 3], device=DEV)
    base, hbase = y.clone(), h.clone()
    mxq.linear(x, w, base, workspace=ws)
    mxq.gated_linear(x, w, hbase, workspace=ws)
    assert bool(torch.isfinite(base).all()) and bool(torch.isfinite(hbase).all())
    for bad in (float("nan"), float("inf")):
        xb, wb = x.clone(), w.clone()
        xb[t, H // 3], wb[f, H // 5] = float("nan"), float("nan")
        mxq.linear(xb, wb, y, workspace=ws)
        only(y, base, t, f, "y")
        mxq.gated_linear(xb, wb, h, workspace=ws)
        only(h, hbase, t, f, "h")  # f is one of the gate's rows
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        dx0, dw0 = torch.empty_like(x), torch.empty_like(w)
        mxq.linear_backward(x, w, dy, dx0, dw0, activation=SILU, z=z, workspace=ws)
        db = dy.clone()
        db[t, f] = bad  # row t of dx, row f of dw
        zb = z.clone()
        zb[t, f] = 1.0
        mxq.linear_backward(x, w, db, dx, dw, activation=SILU, z=zb, workspace=ws)
        only(dx, dx0, t, none, "dx")
        only(dw, dw0, f, none, "dw")
    zero = x * 0
    wz = w.clone()
    wz[:, H // 2] = float("inf")  # 0 times infinity: NaN everywhere, as the sum of products has it
    mxq.linear(zero, wz, y, workspace=ws)
    assert bool(torch.isnan(y).all())


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_two_runs_and_another_stream_give_the_same(n):
    T, H, N = SIZES[n]
    first, db, _ = calls(T, H, N, "gelu", 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, db2, _ = calls(T, H, N, "gelu", 5)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    assert torch.equal(db, db2)


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_captured_calls_that_share_a_workspace(n):
    """Two graphs with one workspace, replayed in turn with the program's own calls between them, on new inputs."""
    T, H, N = SIZES[n]
    x, w, dy = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H)), rn(T, N, seed=3)
    ws = bytes_(max(f(T, H, n, k) for f, n in ((mxq.linear_workspace, N), (mxq.gated_linear_workspace, N // 2)) for k in (0, 1)))

    def forward(o):
        mxq.linear(x, w, o[0], activation=GELU, z=o[1], workspace=ws)
        mxq.gated_linear(x, w, o[2], z=o[3], workspace=ws)

    def backward(o):
        mxq.linear_backward(x, w, dy, o[4], o[5], o[6], GELU, o[1], workspace=ws)
        mxq.gated_linear_backward(x, w, dy[:, :N // 2], o[7], o[8], z=None, workspace=ws)

    make = lambda: [torch.zeros(s, dtype=d, device=DEV) for s, d in (
        ((T, N), BF), ((T, N), BF), ((T, N // 2), BF), ((T, N), BF), ((T, H), BF), ((N, H), BF), ((N,), F32), ((T, H), BF),
        ((N, H), F32))]
    a, b = make(), make()
    forward(a), backward(a)  # before the capture, as a program would
    graphs = []
    for f in (forward, backward):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(a)
        graphs.append(g)
    for turn in range(3):
        for t, seed in ((x, 10), (dy, 20)):
            t.copy_(rn(*t.shape, seed=seed + turn))
        for t in a:
            t.fill_(9.0)
        ws.fill_(255)
        graphs[0].replay()
        forward(b)
        graphs[1].replay()
        backward(b)
        torch.cuda.synchronize()
        for p, q in zip(a, b):
            assert torch.equal(p, q)


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_gradients_one_by_one(n):
    T, H, N = SIZES[n]
    x, w, dy = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H)), rn(T, N, seed=3)
    z, add, old = rn(T, N, seed=4), rn(T, H, seed=5), rn(N, H, seed=6, dtype=F32)
    ws = bytes_(max(f(T, H, n, 1) for f, n in ((mxq.linear_workspace, N), (mxq.gated_linear_workspace, N // 2))))
    for a in ("none", "gelu_tanh"):
        z64 = z.double()
        dz = dy.double() * (1.0 if a == "none" else slope(z64, a))
        err = dz.abs() * (0.0 if a == "none" else 2.0 ** -8) + dy.double().abs() * 2.0 ** -20
        for take in ("x", "w", "b", "xb", "wb"):
            dx = torch.empty_like(x) if "x" in take else None
            dw = old.clone() if "w" in take else None
            db = rn(N, seed=8, dtype=F32) if "b" in take else None
            b0 = None if db is None else db.double()
            mxq.linear_backward(x if "w" in take else x * float("nan"), w if "x" in take else w * float("nan"), dy, dx, dw, db,
                                ACTS[a], None if a == "none" else z, None if dx is None else add, True, ws)
            gradients(dz, err, x, w, dx, dw, None if dx is None else add, None if dw is None else old)
            if db is not None:
                near(db, dz.sum(0) + b0, (dz.abs() + dy.double().abs() * 2.0 ** -20).sum(0) * (T + 2) * 2.0 ** -23
                     + dy.double().abs().sum(0) * 2.0 ** -20 + b0.abs() * 2.0 ** -23, "dbias")
    I = N // 2
    g, u, dh = z[:, :I].double(), z[:, I:].double(), dy[:, :I].double()
    dz = torch.cat([dh * u * slope(g, "silu"), dh * act(g, "silu")], 1)
    err = dz.abs() * 2.0 ** -8 + torch.cat([dh * u, dh * g], 1).abs() * 2.0 ** -19
    for take in ("x", "w"):
        dx = torch.empty_like(x) if "x" in take else None
        dw = torch.empty_like(w) if "w" in take else None
        mxq.gated_linear_backward(x, w, dy[:, :I], dx, dw, z=z, workspace=ws)
        gradients(dz, err, x, w, dx, dw, None, None)


@pytest.mark.parametrize("T", [2, 40, 200])
@pytest.mark.parametrize("name", ["none", "silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(name, T):
    """L(x + e d) - L(x - e d) = 2 e <dx, d> up to the third order, L the sum of y dy (h dh), y in binary32.  d is the sign of dx
    (of dw), so that all terms add up; x, w and the steps are whole multiples of powers of two that bf16 holds.
    The third derivatives of the activations stay below 2, their second ones below 1.2, their first below 1.2."""
    H, N = 64, 48
    x = (rn(T, H, seed=1, dtype=F32) * 16).round().clamp(-56, 56).div(16).to(BF)     # multiples of 1/16 up to 3.5
    w = (rn(N, H, seed=2, dtype=F32) * 16).round().clamp(-56, 56).div(128).to(BF)    # of 1/128
    dy, e = rn(T, N, seed=3), {"x": 2.0 ** -6, "w": 2.0 ** -9}
    ws = bytes_(max(f(T, H, n, k) for f, n in ((mxq.linear_workspace, N), (mxq.gated_linear_workspace, N // 2)) for k in (0, 1)))
    z, dx, dw = torch.empty(T, N, dtype=BF, device=DEV), torch.empty_like(x), torch.empty(N, H, device=DEV)
    y = torch.empty(T, N, device=DEV)
    mxq.linear(x, w, y, activation=ACTS[name], z=z, workspace=ws)
    mxq.linear_backward(x, w, dy, dx, dw, activation=ACTS[name], z=z, workspace=ws)
    for which, grad in (("x", dx), ("w", dw)):
        d = torch.where(grad >= 0, 1.0, -1.0)
        step = e[which]
        ends = []
        for sign in (1, -1):
            xs, ws_ = (x.float() + sign * step * d, w.float()) if which == "x" else (x.float(), w.float() + sign * step * d)
            assert torch.equal(xs, xs.to(BF).float()) and torch.equal(ws_, ws_.to(BF).float())
            mxq.linear(xs.to(BF), ws_.to(BF), y, activation=ACTS[name], workspace=ws)
            ends.append((y.double() * dy.double()).sum())
        got, want = float(grad.double().abs().sum()), float(ends[0] - ends[1]) / (2 * step)
        dz = mm(d, w) if which == "x" else mm(x, d)  # z's change for a step of 1
        dy64 = dy.double().abs()
        third = 0.0 if name == "none" else float((dy64 * dz.abs() ** 3).sum()) * 2.0 * step ** 2 / 6
        sum_err = sums(x, w)[1] * 1.3 + 2.0 ** -20 * mm(x, w).abs() + 2.0 ** -23 * mm(x, w).abs()
        forward = float((dy64 * sum_err).sum()) / step
        # z in bf16 (slope off by at most 1.2 half steps), dz in bf16, dx in bf16
        held = 0.0 if name == "none" else float((dy64 * (1.2 * 2.0 ** -8 + 1.2 * mm(x, w).abs() * 2.0 ** -8) * dz.abs()).sum())
        tol = third + forward + held + got * 2.0 ** -8 + float((dy64 * dz.abs()).sum()) * 2.0 ** -18
        assert abs(got - want) <= tol, (got, want, tol)
        assert tol < 0.25 * got  # says something


def test_gated_gradients_against_differences():
    """As above; the third derivative of act(g) u along (dg, du) is act''' dg^3 u + 3 act'' dg^2 du.  h is rounded to bf16, its
    error a random one of half a step at most: counted in full."""
    T, H, I = 60, 64, 24
    x = (rn(T, H, seed=1, dtype=F32) * 16).round().clamp(-56, 56).div(16).to(BF)
    w = (rn(2 * I, H, seed=2, dtype=F32) * 16).round().clamp(-56, 56).div(128).to(BF)
    dh = rn(T, I, seed=3)
    ws = bytes_(max(mxq.gated_linear_workspace(T, H, I, k) for k in (0, 1)))
    z64 = mm(x, w)
    g, u = z64[:, :I], z64[:, I:]
    for kept in (True, False):
        z, h = torch.empty(T, 2 * I, dtype=BF, device=DEV), torch.empty(T, I, dtype=BF, device=DEV)
        dx, dw = torch.empty_like(x), torch.empty(2 * I, H, device=DEV)
        mxq.gated_linear(x, w, h, z=z, workspace=ws)
        mxq.gated_linear_backward(x, w, dh, dx, dw, z=z if kept else None, workspace=ws)
        for which, grad, step in (("x", dx, 2.0 ** -6), ("w", dw, 2.0 ** -9)):
            d = torch.where(grad >= 0, 1.0, -1.0).double()
            # differences of the formula in 64 bits: the kernel's own h, in bf16, is too coarse for a small step
            ends = []
            for sign in (1, -1):
                zz = mm(x.double() + sign * step * d, w) if which == "x" else mm(x, w.double() + sign * step * d)
                ends.append((act(zz[:, :I], "silu") * zz[:, I:] * dh.double()).sum())
            got, want = float(grad.double().abs().sum()), float(ends[0] - ends[1]) / (2 * step)
            dz = (mm(d, w) if which == "x" else mm(x, d)).abs()
            dg, du = dz[:, :I], dz[:, I:]
            a = dh.double().abs()
            third = float((a * (2 * dg ** 3 * u.abs() + 3.6 * dg ** 2 * du)).sum()) * step ** 2 / 6
            parts = a * (1.2 * u.abs() * dg + (g.abs() + 0.3) * du)  # magnitudes of what dz is made of
            held = float((parts + a * (1.2 * g.abs() * u.abs() * dg + 1.2 * g.abs() * du)).sum()) * 2.0 ** -8 * (2.1 if kept else 1.05)
            tol = third + held + got * 2.0 ** -8 + float(parts.sum()) * 2.0 ** -18
            assert abs(got - want) <= tol, (got, want, tol, kept, which)


@pytest.mark.parametrize("T,H,N", [(300000, 64, 16384), (2, 16384, 270336), (40, 16384, 270336), (140, 65536, 65600),
                                   (1 << 19, 8200, 64)])
def test_matrices_of_more_than_2_to_the_32_bytes(T, H, N):
    """x, w, y and dw past 2^32 bytes or elements, looked at where the offsets are large."""
    g = torch.Generator(device=DEV).manual_seed(1)

    def big(r, c, std=1.0):
        t = torch.empty(r, c, dtype=BF, device=DEV)
        for k in range(0, r, 1 << 14):
            t[k:k + (1 << 14)].normal_(0.0, std, generator=g)
        return t
    x, w, dy = big(T, H), big(N, H, 1 / math.sqrt(H)), big(T, N)
    ws = bytes_(max(mxq.linear_workspace(T, H, N, k) for k in (0, 1)))
    rows = torch.tensor(sorted({0, T // 2, T - 2, T - 1} - {-1}), device=DEV)
    cols = torch.tensor(sorted({0, 5, N // 2, N - 9, N - 1}), device=DEV)
    y = torch.empty(T, N, dtype=BF, device=DEV)
    mxq.linear(x, w, y, activation=ACTS["relu"], residual=dy, workspace=ws)
    want, tol = sums(x[rows], w)
    near(y[rows], torch.relu(want) + dy[rows].double(), tol * 1.2 + 2.0 ** -22 * (want.abs() + dy[rows].double().abs()), "rows")
    want, tol = sums(x, w[cols])
    near(y[:, cols], torch.relu(want) + dy[:, cols].double(),
         tol * 1.2 + 2.0 ** -22 * (want.abs() + dy[:, cols].double().abs()), "columns")
    del y
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device=DEV)
    mxq.linear_backward(x, w, dy, dx, dw, db, workspace=ws)
    few = dy[:, cols].double()
    near(db[cols], few.sum(0), few.abs().sum(0) * (T + 2) * 2.0 ** -24, "dbias")
    gradients(few, few.abs() * 0, x, w[cols], None, dw[cols], None, None)
    a = torch.empty(len(rows), H, dtype=F64, device=DEV)
    m = torch.empty_like(a)
    for k in range(0, H, 4096):
        part = w[:, k:k + 4096].double()
        a[:, k:k + 4096] = torch.mm(dy[rows].double(), part)
        m[:, k:k + 4096] = torch.mm(dy[rows].double().abs(), part.abs())
    near(dx[rows], a, m * ((N / 32 + 40) * SUM), "dx")


@pytest.mark.parametrize("T,H,N", [(16, 4096, 11272), (32, 4104, 11272), (50, 2880, 16384), (128, 4096, 11272), (90, 11272, 4096),
                                   (17, 32768, 1416)])
def test_gradients_of_few_tokens_and_large_weights(T, H, N):
    x, w = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H))
    dy, add, old = rn(T, N, seed=3), rn(T, H, seed=4), rn(N, H, seed=5, dtype=F32)
    ws = bytes_(mxq.linear_workspace(T, H, N, True))
    for more in (False, True):
        dx, dw = torch.empty_like(x), old.clone()
        mxq.linear_backward(x, w, dy, dx, dw, add=add if more else None, accumulate=more, workspace=ws)
        gradients(dy.double(), dy.double() * 0, x, w, dx, dw, add if more else None, old if more else None)


@pytest.mark.parametrize("T,H,N", [(2048, 2056, 4112), (1000, 4096, 4112), (600, 2880, 6000), (4104, 1032, 2048), (1100, 1416, 10000),
                                   (2000, 2880, 1008), (300, 8200, 1040)])
def test_both_gradients_in_one_launch(T, H, N):
    """Middle sizes, whose products share a launch of large or of small tiles, cut or not, the bias's sums with them; and the
    same products each on its own."""
    x, w = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H))
    dy, add, old = rn(T, N, seed=3), rn(T, H, seed=4), rn(N, H, seed=5, dtype=F32)
    ws = bytes_(mxq.linear_workspace(T, H, N, True))
    dy64 = dy.double()
    for more in (False, True):
        dx, dw, db = torch.empty_like(x), old.clone() if more else torch.empty_like(w), torch.ones(N, device=DEV)
        mxq.linear_backward(x, w, dy, dx, dw, db, add=add if more else None, accumulate=more, workspace=ws)
        gradients(dy64, dy64 * 0, x, w, dx, dw, add if more else None, old if more else None)
        near(db, dy64.sum(0) + more, (dy64.abs().sum(0) + more) * (T + 2) * 2.0 ** -24, "dbias")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    mxq.linear_backward(x, w, dy, dx=dx, workspace=ws)
    mxq.linear_backward(x, w, dy, dw=dw, workspace=ws)
    gradients(dy64, dy64 * 0, x, w, dx, dw, None, None)
    z, gx, gw = rn(T, N, seed=6), torch.empty_like(x), torch.empty_like(w)
    I = N // 2
    ws = bytes_(mxq.gated_linear_workspace(T, H, I, True))
    mxq.gated_linear_backward(x, w, dy[:, :I], gx, gw, z=z, add=add, workspace=ws)
    g, u, dh = z[:, :I].double(), z[:, I:].double(), dy64[:, :I]
    dz = torch.cat([dh * u * slope(g, "silu"), dh * act(g, "silu")], 1)
    gradients(dz, dz.abs() * 2.0 ** -8 + torch.cat([dh * u, dh * g], 1).abs() * 2.0 ** -19, x, w, gx, gw, add, None)


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("T", [1, 33, 300])
def test_a_block_and_its_update(T, eight):
    """y = x + act-gated x w1 through w2, its gradients, their norm and the update, as a training step calls them: the
    gradients against the formulas, every rounding on the way followed as an interval; the parameters against the
    update with the gradients that came out, clipped."""
    H, I = 264, 328
    x, dy = rn(T, H, seed=1), rn(T, H, seed=2)
    w1, w2 = rn(2 * I, H, seed=3, std=1 / 16, dtype=F32), rn(H, I, seed=4, std=1 / 18, dtype=F32)
    c1, c2 = w1.to(BF), w2.to(BF)
    b2 = rn(H, seed=5, dtype=F32)
    params = [w1, w2, b2]
    grads = [torch.zeros_like(t) for t in params]
    if eight:
        codes = [[torch.zeros(t.numel(), dtype=torch.uint8, device=DEV) for t in params] for _ in range(2)]
        scales = [[torch.zeros(-(-t.numel() // 128), device=DEV) for t in params] for _ in range(2)]
        update = mxq.AdamW(params, grads, *codes, *scales, copies=[c1, c2, None], decay=[True, True, False])
    else:
        moments = [[torch.zeros_like(t) for t in params] for _ in range(2)]
        update = mxq.AdamW(params, grads, *moments, copies=[c1, c2, None], decay=[True, True, False])
    z, h, y = (torch.empty(T, n, dtype=BF, device=DEV) for n in (2 * I, I, H))
    dh, dx, norm = torch.empty_like(h), torch.empty_like(x), torch.zeros(1, device=DEV)
    ws = bytes_(max(max(mxq.gated_linear_workspace(T, H, I, k), mxq.linear_workspace(T, I, H, k)) for k in (0, 1)))
    every = mxq.GradientSet(grads)
    rate, betas, eps, wd, most = 0.01, (0.9, 0.95), 1e-8, 0.1, 0.5
    before, b1, b2c = [t.double() for t in params], c1.double(), c2.double()
    mxq.gated_linear(x, c1, h, z=z, workspace=ws)
    mxq.linear(h, c2, y, bias=b2, residual=x, workspace=ws)
    mxq.linear_backward(h, c2, dy, dh, grads[1], grads[2], workspace=ws)
    mxq.gated_linear_backward(x, c1, dh, dx, grads[0], z=z, add=dy, workspace=ws)
    every.norm(norm)
    update.step(1, rate, betas, eps, wd, norm=norm, max_norm=most, seed=3)
    # the block in 64 bits
    zz, ztol = sums(x, b1.to(BF))
    g, u = zz[:, :I], zz[:, I:]
    near(z, zz, ztol, "z")
    h64 = act(g, "silu") * u
    eh = 1.2 * (ztol[:, :I] * u.abs() + ztol[:, I:] * g.abs()) + 2.0 ** -19 * h64.abs() + 2.0 ** -8 * h64.abs()
    near(h, h64, eh, "h")
    y64 = torch.mm(h64, b2c.t().contiguous()) + before[2] + x.double()
    ey = torch.mm(eh + h64.abs() * ((I / 32 + 40) * SUM), b2c.abs().t().contiguous()) + 2.0 ** -22 * (y64.abs() + x.double().abs())
    near(y, y64, ey, "y")
    dy64 = dy.double()
    dh64 = torch.mm(dy64, b2c)
    edh = torch.mm(dy64.abs(), b2c.abs()) * ((H / 32 + 40) * SUM) + 2.0 ** -8 * dh64.abs()
    near(grads[1], torch.mm(dy64.t().contiguous(), h64),
         torch.mm(dy64.abs().t().contiguous(), eh + h64.abs() * ((T / 32 + 40) * SUM)), "dw2")
    near(grads[2], dy64.sum(0), dy64.abs().sum(0) * (T + 2) * 2.0 ** -24, "db2")
    eg, eu = ztol[:, :I] + 2.0 ** -8 * g.abs(), ztol[:, I:] + 2.0 ** -8 * u.abs()  # z is held in bf16
    s, s1 = act(g, "silu"), slope(g, "silu")
    dg, du = dh64 * u * s1, dh64 * s
    # |silu'| <= 1.1, |silu''| <= 0.5; products of two errors: 2^-6 more
    edg = (edh * (u * s1).abs() + dh64.abs() * (eu * s1.abs() + 0.5 * eg * u.abs())) * (1 + 2.0 ** -6) + dh64.abs() * eg * eu
    edu = (edh * s.abs() + dh64.abs() * 1.1 * eg) * (1 + 2.0 ** -6)
    dz = torch.cat([dg, du], 1)
    edz = torch.cat([edg + edh * eu, edu], 1)
    edz = edz + (dz.abs() + edz) * 2.0 ** -8 + torch.cat([dh64 * u, dh64 * g], 1).abs() * 2.0 ** -19
    gradients(dz, edz, x, b1.to(BF), dx, grads[0], dy, None)
    # the norm and the update, of these gradients
    n64 = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    assert abs(float(norm) - n64) <= 2.0 ** -23 * n64
    coef = min(1.0, most / (n64 + 1e-6))
    assert coef < 1.0
    for k, (p, q, t) in enumerate(zip(params, before, grads)):
        gr = t.double() * coef
        m, v = (1 - betas[0]) * gr, (1 - betas[1]) * gr ** 2
        step = rate * (m / (1 - betas[0])) / ((v / (1 - betas[1])).sqrt() + eps)
        want = q * (1 - rate * wd * (k < 2)) - step
        # some ten roundings of the quotient, each 2^-24; gradients near 2^-60 do not occur
        near(p, want, q.abs() * 2.0 ** -22 + step.abs() * 2.0 ** -19 + 1e-12, f"params[{k}]")
    assert torch.equal(c1, w1.to(BF)) and torch.equal(c2, w2.to(BF))


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own, and the update of one behind the products of the other."""
    T, H, N = 300, 1032, 2064
    x, w = rn(T, H, seed=1), rn(N, H, seed=2, std=1 / math.sqrt(H))
    dy = [rn(T, N, seed=3 + k) for k in range(2)]
    n = mxq.linear_workspace(T, H, N, True)

    def call(k, ws, dx, dw, db, p, s):
        for _ in range(5):
            mxq.linear_backward(x, w, dy[k], dx, dw, db, workspace=ws)
            s.step(1, 0.01, norm=None)

    def buffers():
        p = [torch.ones(N, H, device=DEV)]
        dw = torch.empty(N, H, device=DEV)
        s = mxq.AdamW(p, [dw], [torch.zeros_like(dw)], [torch.zeros_like(dw)])
        return bytes_(n), torch.empty_like(x), dw, torch.empty(N, device=DEV), p, s
    one = [buffers() for _ in range(2)]
    for k in range(2):
        call(k, *one[k])
    torch.cuda.synchronize()
    two, streams = [buffers() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            call(k, *two[k])
    torch.cuda.synchronize()
    for a, b in zip(one, two):
        for p, q in zip(a[1:4], b[1:4]):
            assert torch.equal(p, q)
        assert torch.equal(a[4][0], b[4][0])


def test_an_update_beyond_2_to_the_31_elements():
    """The elements about 2^31 and the last ones of a large tensor, bit for bit as in a small one."""
    n, k = (1 << 31) + 5000, 3000
    p, g = (torch.zeros(n, dtype=BF, device=DEV) for _ in range(2))
    m, v = (torch.zeros(n, device=DEV) for _ in range(2))
    places = [slice(0, k), slice((1 << 31) - k // 2, (1 << 31) + k // 2), slice(n - k, n)]
    small = []
    for i, at in enumerate(places):
        p[at], g[at] = rn(k, seed=2 * i), rn(k, seed=2 * i + 1)
        small.append([p[at].clone(), g[at].clone(), m[at].clone(), v[at].clone()])
    big = mxq.AdamW([p], [g], [m], [v])
    few = mxq.AdamW(*([s[j] for s in small] for j in range(4)))
    norm, want = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    mxq.GradientSet([g]).norm(norm)
    mxq.GradientSet([s[1] for s in small]).norm(want)
    assert torch.allclose(norm, want, rtol=2.0 ** -22, atol=0.0)
    for t in (1, 2):
        big.step(t, 0.01, norm=norm, max_norm=0.5)
        few.step(t, 0.01, norm=norm, max_norm=0.5)
    for at, s in zip(places, small):
        for a, b in zip((p, g, m, v), s):
            assert torch.equal(a[at], b)
    between = slice((1 << 31) - 100000, (1 << 31) - k)
    assert not bool(p[between].any()) and not bool(m[between].any())
