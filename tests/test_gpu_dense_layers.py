"""Linear and gated layers and their gradients against their definitions in 64 bits (GPU).

Tolerances, from the roundings that the kernels make:
  a sum of K exact products of bf16 values: an MFMA adds 32 of them and one accumulator, each addition off by at most
    2^-23 of what it adds up, so at most (K / 32 + 40) 2^-23 of the sum of the products' magnitudes
  an activation in binary32: at most 2^-20 of |z| (its value) or of 1 (its derivative), and 1.2 times z's own error
  a rounding to bf16: 2^-8 of the value; to binary32: 2^-24
  gradients before the products: held in bf16, 2^-8 of each entry
"""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64 = "cuda", torch.bfloat16, torch.float32, torch.float64
ACTS = {"none": mxq.ACT_NONE, "relu": mxq.ACT_RELU, "silu": mxq.ACT_SILU, "gelu": mxq.ACT_GELU,
        "gelu_tanh": mxq.ACT_GELU_TANH}
SUM, ACT, HALF = 2.0 ** -23, 2.0 ** -20, {BF: 2.0 ** -8, F32: 2.0 ** -24}


def act(z, name):
    if name == "gelu_tanh":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[name](z)


def slope(z, name):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(act(z, name).sum(), z)[0]


def rn(*shape, seed, std=1.0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def mm(a, b):
    """a b^T in 64 bits."""
    return torch.mm(a.double(), b.double().t().contiguous())


def sums(a, b):
    """a b^T and the bound of a binary32 sum of its products."""
    return mm(a, b), mm(a.abs(), b.abs()) * ((a.shape[1] / 32 + 40) * SUM)


def near(got, want, tol, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= tol + HALF[got.dtype] * want.abs() + 1e-38)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(), float((off / (tol + 1e-38)).max()), bad.nonzero()[:4].tolist())


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


# tokens, hidden, features: the paths for few rows, every tile, splits of the sum, partial tiles
SIZES = [(1, 8, 8), (1, 264, 1000), (1, 4096, 4096), (2, 7176, 264), (3, 2056, 40), (4, 1032, 8200), (5, 200, 24584),
         (31, 8192, 8200), (40, 64, 28680), (64, 5416, 8328), (60, 1032, 1000), (100, 264, 24600), (128, 8200, 8192), (16, 520, 248), (17, 136, 72), (23, 2880, 520),
         (33, 64, 2056), (65, 1096, 200), (130, 520, 136), (257, 72, 520), (300, 4096, 1032), (700, 264, 4104),
         (1030, 1000, 2056), (2048, 512, 4096), (5000, 200, 3096),
         (1024, 4096, 14336), (2011, 2880, 5000), (1500, 1416, 10000)]


def forward(T, H, N, name, bias, residual, keep, out, seed):
    x, w = rn(T, H, seed=seed), rn(N, H, seed=seed + 1, std=1 / math.sqrt(H))
    b = rn(N, seed=seed + 2, std=0.5, dtype=F32) if bias else None
    r = rn(T, N, seed=seed + 3, dtype=out) if residual else None
    y, z = torch.empty(T, N, dtype=out, device=DEV), torch.empty(T, N, dtype=BF, device=DEV) if keep else None
    mxq.linear(x, w, y, bias=b, activation=ACTS[name], residual=r, z=z, workspace=bytes_(mxq.linear_workspace(T, H, N)))
    want, tol = sums(x, w)
    if bias:
        want += b.double()
        tol += want.abs() * 2.0 ** -24
    if keep:
        near(z, want, tol, "z")
    tol = 1.2 * tol + ACT * want.abs()
    want = act(want, name)
    if residual:
        want += r.double()
        tol += (want.abs() + r.double().abs()) * 2.0 ** -24
    near(y, want, tol, "y")


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_linear(n):
    T, H, N = SIZES[n]
    names = list(ACTS)
    forward(T, H, N, names[n % 5], n % 2 == 0, n % 3 == 0, n % 4 < 2, BF if n % 7 < 4 else F32, 10 * n)
    forward(T, H, N, names[(n + 2) % 5], n % 2 == 1, n % 3 != 0, n % 4 >= 2, F32 if n % 7 < 4 else BF, 10 * n + 5)


@pytest.mark.parametrize("name", list(ACTS))
@pytest.mark.parametrize("T,H,N", [(2, 64, 40), (150, 72, 264)])
def test_activations_over_their_range(name, T, H, N):
    """Sums from 1e-4 to 60 of either sign."""
    x = rn(T, H, seed=1)
    w = rn(N, H, seed=2, std=1 / math.sqrt(H)) * torch.logspace(-3, 1.3, N, device=DEV).to(BF)[:, None]
    y, z = torch.empty(T, N, device=DEV), torch.empty(T, N, dtype=BF, device=DEV)
    mxq.linear(x, w, y, activation=ACTS[name], z=z, workspace=bytes_(mxq.linear_workspace(T, H, N)))
    want, tol = sums(x, w)
    near(z, want, tol)
    near(y, act(want, name), 1.2 * tol + ACT * want.abs())
    dy = rn(T, N, seed=3)
    db, dx = torch.empty(N, device=DEV), torch.empty(T, H, dtype=BF, device=DEV)
    mxq.linear_backward(x, w, dy, dx, dbias=db, activation=ACTS[name], z=z,
                        workspace=bytes_(mxq.linear_workspace(T, H, N, True)))
    d = dy.double() * slope(z.double(), name)
    near(db, d.sum(0), dy.double().abs().sum(0) * (ACT + T * 2.0 ** -23))


def gradients(dz, dzerr, x, w, dx, dw, add, old, tol_z=None):
    """Checks dx and dw against dz (64 bits), whose error before the products is at most dzerr."""
    T, N = dz.shape
    if dx is not None:
        want = torch.mm(dz, w.double())
        tol = torch.mm(dzerr + dz.abs() * ((N / 32 + 40) * SUM), w.double().abs())
        if add is not None:
            want += add.double()
            tol += want.abs() * 2.0 ** -24
        near(dx, want, tol, "dx")
    if dw is not None:
        want = torch.mm(dz.t().contiguous(), x.double())
        tol = torch.mm((dzerr + dz.abs() * ((T / 32 + 40) * SUM)).t().contiguous(), x.double().abs())
        if old is not None:
            want += old.double()
            tol += want.abs() * 2.0 ** -24
        near(dw, want, tol, "dw")


@pytest.mark.parametrize("n", range(len(SIZES)), ids=["x".join(map(str, s)) for s in SIZES])
def test_linear_backward(n):
    T, H, N = SIZES[n]
    names, seed = list(ACTS), 100 + 10 * n
    for k, name in enumerate((names[n % 5], names[(n + 3) % 5])):
        x, w = rn(T, H, seed=seed), rn(N, H, seed=seed + 1, std=1 / math.sqrt(H))
        z, dy = rn(T, N, seed=seed + 2), rn(T, N, seed=seed + 3)
        out = (BF, F32)[(n + k) % 2]
        add = rn(T, H, seed=seed + 4) if (n + k) % 3 else None
        old, oldb = rn(N, H, seed=seed + 5, dtype=out), rn(N, seed=seed + 6, dtype=F32)
        dx, dw, db = torch.empty(T, H, dtype=BF, device=DEV), old.clone(), oldb.clone()
        accumulate = (n + k) % 4 < 2
        mxq.linear_backward(x, w, dy, dx, dw, db, activation=ACTS[name], z=z if name != "none" else None, add=add,
                            accumulate=accumulate, workspace=bytes_(mxq.linear_workspace(T, H, N, True)))
        dz = dy.double() * slope(z.double(), name)
        held = dy.double().abs() * ACT + (dz.abs() * HALF[BF] if name != "none" else 0.0)
        gradients(dz, held, x, w, dx, dw, add, old if accumulate else None)
        want = dz.sum(0) + (oldb.double() if accumulate else 0.0)
        near(db, want, (dy.double().abs() * ACT + dz.abs() * (T * 2.0 ** -23)).sum(0) + want.abs() * 2.0 ** -24, "dbias")


GATED = [(1, 8, 8), (1, 4096, 264), (1, 5128, 1000), (2, 264, 24), (4, 520, 4104), (6, 520, 12296), (25, 4104, 5608),
         (33, 72, 12360), (50, 8200, 4104), (110, 520, 14344), (16, 2880, 200), (17, 520, 40), (48, 2048, 1000), (65, 72, 136),
         (130, 520, 264), (300, 1096, 1032), (700, 264, 2056), (2048, 512, 2048), (1100, 4096, 1544), (5000, 200, 1560), (2011, 2880, 5000), (1500, 1416, 7000)]
GACTS = ["silu", "gelu", "gelu_tanh", "relu", "none"]


def pair(z):
    return z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]


@pytest.mark.parametrize("n", range(len(GATED)), ids=["x".join(map(str, s)) for s in GATED])
def test_gated_linear(n):
    T, H, I = GATED[n]
    name = GACTS[n % 5]
    x, w = rn(T, H, seed=n), rn(2 * I, H, seed=n + 50, std=1 / math.sqrt(H))
    h, z = torch.empty(T, I, dtype=BF, device=DEV), torch.empty(T, 2 * I, dtype=BF, device=DEV) if n % 2 else None
    mxq.gated_linear(x, w, h, activation=ACTS[name], z=z, workspace=bytes_(mxq.gated_linear_workspace(T, H, I)))
    want, tol = sums(x, w)
    if z is not None:
        near(z, want, tol, "z")
    (g, u), (tg, tu) = pair(want), pair(tol)
    a = act(g, name)
    ta = 1.2 * tg + ACT * g.abs()
    near(h, a * u, ta * u.abs() + tu * a.abs() + ta * tu + 2.0 ** -23 * (a * u).abs(), "h")


@pytest.mark.parametrize("n", range(len(GATED)), ids=["x".join(map(str, s)) for s in GATED])
@pytest.mark.parametrize("kept", [True, False], ids=["kept", "again"])
def test_gated_linear_backward(n, kept):
    T, H, I = GATED[n]
    name, seed = GACTS[(n + kept) % 5], 300 + 10 * n
    x, w, dh = rn(T, H, seed=seed), rn(2 * I, H, seed=seed + 1, std=1 / math.sqrt(H)), rn(T, I, seed=seed + 2)
    z = rn(T, 2 * I, seed=seed + 3) if kept else None
    out = (BF, F32)[n % 2]
    add = rn(T, H, seed=seed + 4) if n % 3 else None
    old = rn(2 * I, H, seed=seed + 5, dtype=out)
    dx, dw = torch.empty(T, H, dtype=BF, device=DEV), old.clone()
    mxq.gated_linear_backward(x, w, dh, dx, dw, activation=ACTS[name], z=z, add=add, accumulate=n % 4 < 2,
                              workspace=bytes_(mxq.gated_linear_workspace(T, H, I, True)))
    v, tv = (z.double(), torch.zeros(T, 2 * I, dtype=F64, device=DEV)) if kept else sums(x, w)
    (g, u), (tg, tu) = pair(v), pair(tv)
    d, a, s = dh.double(), act(g, name), slope(g, name)
    # act'' is below 1.2 for every activation but the ReLU, whose slope jumps where the gate's sign is in doubt
    ts = ACT + 1.2 * tg if name != "relu" else (g.abs() <= tg).double()
    dz = torch.cat([d * u * s, d * a], 1)
    err = torch.cat([d.abs() * (u.abs() * ts + tu * s.abs() + tu * ts), d.abs() * (1.2 * tg + ACT * g.abs())], 1)
    gradients(dz, err + (dz.abs() + err) * HALF[BF], x, w, dx, dw, add, old if n % 4 < 2 else None)
