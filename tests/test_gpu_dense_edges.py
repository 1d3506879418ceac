"""Activations of linear and gated layers at the ends of their range against their definitions in 64 bits (GPU): slopes at
large finite arguments, and the lower tail.

The arguments reach the kernels exactly: a kept z is given as it is, and a product has one term (all others are 0 times a
finite value).
"""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from test_gpu_dense_layers import ACTS, BF, DEV, F32, bytes_, near

pytestmark = pytest.mark.gpu
# either sign, up to bf16's largest value; squares pass binary32's range from 1.8e19 on
LARGE = [s * v for v in (12.0, 20.0, 89.0, 128.0, 1e4, 1e10, 1e19, 3e19, 6e19, 1e20, 1e30, 3.3895e38) for s in (1, -1)]


def cdf(z):
    """Phi(z), its lower tail with its precision."""
    return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))


def value_and_slope(z, name):
    """In 64 bits; the sigmoids of both signs by their own exponentials, so that no difference cancels."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if name == "gelu":
        p = cdf(z)
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    u, du = z, torch.ones_like(z)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    p, n = torch.sigmoid(u), torch.sigmoid(-u)
    return z * p, p + z * p * n * du


@pytest.mark.parametrize("name", list(ACTS))
def test_slopes_at_large_arguments(name):
    """dbias of one token is dy times the slope, of 2 each: 0 or 1 but for less than 2^-20 at these arguments."""
    z = torch.tensor(LARGE, device=DEV).to(BF)[None]
    N, H = z.shape[1], 8
    x, w, dy = torch.zeros(1, H, dtype=BF, device=DEV), torch.zeros(N, H, dtype=BF, device=DEV), torch.full_like(z, 2.0)
    db = torch.empty(N, device=DEV)
    mxq.linear_backward(x, w, dy, dbias=db, activation=ACTS[name], z=z, workspace=bytes_(mxq.linear_workspace(1, H, N, True)))
    want = value_and_slope(z.double(), name)[1][0]
    assert bool(want.isfinite().all())
    near(db, 2.0 * want, 2.0 ** -19)


@pytest.mark.parametrize("kept", [True, False], ids=["kept", "again"])
@pytest.mark.parametrize("T", [8, 40, 304, 1032])
@pytest.mark.parametrize("name", list(ACTS))
def test_gated_gradients_at_large_arguments(name, T, kept):
    """Token t has the gate LARGE[t] in every feature and an up of 1: dgate = dh act'(gate), dup = dh act(gate).  x holds the gate
    in column 0, and 1 in column 8 + t, where dw's rows therefore hold dgate and dup."""
    I, H = 264, T + 8
    v = torch.tensor([LARGE[t % len(LARGE)] for t in range(T)], device=DEV).to(BF)
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    x[:, 0] = v
    x[torch.arange(T), 8 + torch.arange(T)] = 1.0
    w = torch.zeros(2 * I, H, dtype=BF, device=DEV)
    w[:I, 0] = 1.0
    w[I:, 8:] = 1.0
    z = torch.cat([v[:, None].expand(T, I), torch.ones(T, I, dtype=BF, device=DEV)], 1).contiguous() if kept else None
    dh = torch.full((T, I), 2.0 ** -60, dtype=BF, device=DEV)  # so that dup stays below bf16's largest value
    dw = torch.empty(2 * I, H, device=DEV)
    mxq.gated_linear_backward(x, w, dh, dw=dw, activation=ACTS[name], z=z, workspace=bytes_(mxq.gated_linear_workspace(T, H, I, True)))
    a, d = value_and_slope(v.double(), name)
    # each in bf16 before the products, which are exact, then in binary32; a value's own error 2^-20 of |z|, a slope's 2^-20
    near(dw[:I, 8:], (2.0 ** -60 * d)[None].expand(I, T), 2.0 ** -60 * (2.0 ** -8 * d.abs() + 2.0 ** -20), "dgate")
    near(dw[I:, 8:], (2.0 ** -60 * a)[None].expand(I, T), 2.0 ** -60 * (2.0 ** -8 * a.abs() + 2.0 ** -20 * v.double().abs()), "dup")


def tail(z):
    """A relative bound of Phi(z) in binary32 below 0.  The exponential: its argument z^2 / 2 log2 e from three roundings (of
    z^2, the constant and the product) of half a step, 2^-24 each, so 1.5 z^2 2^-24 of its value.  The fit of Phi's other factor, a
    polynomial of degree 7 in t = 1 / (1 + c |z|): less than 2^-22 + z^2 2^-25.  t itself, off by 1.5 2^-23, counts threefold at
    most (the factor's slope over its value, times t); exp2, the polynomial's steps and the two products: 3.5 2^-23."""
    return 8 * 2.0 ** -23 + 2.0 ** -22 + z * z * (1.5 * 2.0 ** -24 + 2.0 ** -25)


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 16, 48, 130, 512, 2048])
def test_the_lower_tail_of_gelu(T, out):
    """Rounded once: the value is right to its last place where it is small, as far as it is no subnormal."""
    N, H = 2048, 72
    z = -torch.logspace(math.log10(2.0 ** -10), math.log10(12.75), N, device=DEV).to(BF)
    x, w = torch.zeros(T, H, dtype=BF, device=DEV), torch.zeros(N, H, dtype=BF, device=DEV)
    x[:, 5], w[:, 5] = 1.0, z
    y = torch.empty(T, N, dtype=out, device=DEV)
    mxq.linear(x, w, y, activation=mxq.ACT_GELU, workspace=bytes_(mxq.linear_workspace(T, H, N)))
    z = z.double()
    want = (z * cdf(z))[None].expand(T, N)
    near(y, want, want.abs() * (tail(z) + 2.0 ** -23), "y")


def test_the_lower_tail_of_gelus_slope():
    N, H = 2048, 8
    z = -torch.logspace(math.log10(2.0 ** -10), math.log10(12.75), N, device=DEV).to(BF)[None]
    x, w, dy = torch.zeros(1, H, dtype=BF, device=DEV), torch.zeros(N, H, dtype=BF, device=DEV), torch.ones_like(z)
    db = torch.empty(N, device=DEV)
    mxq.linear_backward(x, w, dy, dbias=db, activation=mxq.ACT_GELU, z=z, workspace=bytes_(mxq.linear_workspace(1, H, N, True)))
    z = z[0].double()
    density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    # the terms' bounds, of opposite signs, the density's constant and product, and the sum
    near(db, cdf(z) + z * density, (cdf(z) + z.abs() * density) * (tail(z) + 3 * 2.0 ** -24))
