"""The AdamW step where its definition leaves no room (GPU): clipping by norms near binary32's ends, codes and scales of 8-bit
moments bit for bit, roots of subnormal moments.

h = 2^-24: half a step of binary32, relative."""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from test_gpu_adamw import BF, DEV, E4, E5, F32, U8, chance, h, rn

pytestmark = pytest.mark.gpu


def clipped(g, norm, most):
    """The gradients that a step takes, as it leaves them in m where beta1 is 0 (m = 0 m + 1 g): states of zero."""
    n = g.numel()
    p, m, v, total = (torch.zeros(k, device=DEV) for k in (n, n, n, 1))
    total.fill_(norm)
    mxq.AdamW([p], [g], [m], [v]).step(1, 0.0, (0.0, 0.0), 1e-8, 0.0, norm=total, max_norm=most)
    return m


@pytest.mark.parametrize("most", [1e-30, 1e-6, 1.0, 1e20, 1e38, 1e39])
@pytest.mark.parametrize("norm", [1e-37, 1e-3, 1.0, 1e30, 1e37, 2e38, 3.4e38])
def test_clipping_over_the_whole_range_of_norms(norm, most):
    """min(1, max_norm / (norm + 1e-6)) keeps its precision wherever the products are normal numbers: three roundings of the
    coefficient, one of the product, and the subnormals' step."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    g = rn(4096, gen)
    g *= min(norm, 1e38) / 4096.0
    norm = float(torch.tensor(norm, dtype=F32))
    m = clipped(g, norm, most).double()
    want = g.double() * min(1.0, most / (norm + 1e-6))
    assert bool(((m - want).abs() <= 4 * h * want.abs() + 2.0 ** -149).all()), float(((m - want).abs() / want.abs().clamp(min=1e-44)).max())


def test_an_infinite_norm_leaves_finite_gradients_zero():
    g = torch.tensor([1.0, -2.0, 3e38, 0.0], device=DEV)
    for most in (0.0, 1.0, 1e38, 1e39, 1e300):
        assert bool((clipped(g, float("inf"), most) == 0.0).all()), most
        assert bool(clipped(g, float("nan"), most).isnan().all()), most


@pytest.mark.parametrize("std", [1e-20, 1.0, 1e30])
def test_a_step_clips_as_the_set_does(std):
    """GradientSet.clip's values, whose one rounding is half a step, against a step's: the same but for 5 half steps."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    g = rn(1 << 16, gen) * std * (1e6 if std > 1 else 1.0)
    norm, out = torch.zeros(1, device=DEV), torch.empty_like(g)
    for most in (1e-3, 1.0, 1e33):
        mxq.GradientSet([g], [out]).clip(most, norm)
        m = clipped(g, float(norm), most)
        assert bool(((m.double() - out.double()).abs() <= 6 * h * out.double().abs() + 2.0 ** -148).all()), (std, most)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("p,g", [(F32, F32), (F32, BF), (BF, BF)])
def test_8bit_moments_follow_the_plain_sequence_of_roundings(p, g, clip):
    """Codes and scales bit for bit those of the header's definition, each operation rounded to binary32 (on the CPU, whose
    arithmetic is IEEE's): values over many magnitudes, blocks of zeros, a short last block."""
    n, t, seed, (b1, b2) = 200037, 17, 5, (0.9, 0.99)
    gen = torch.Generator().manual_seed(3)
    size = torch.exp2(torch.randint(-30, 10, (n // 128 + 1, 1), generator=gen).float()).expand(-1, 128).reshape(-1)[:n]
    inner = torch.exp2(-torch.rand(n, generator=gen) * 14)
    grad = (torch.randn(n, generator=gen) * size * inner).to(g)
    grad[1280:1536] = 0.0
    m, v = (torch.randint(0, 256, (n,), generator=gen).to(U8) for _ in range(2))
    m[(m & 0x7F) == 0x7F] = 0          # no NaN
    v = v & 0x7F
    v[v > 0x7B] = 0x7B                 # neither infinity nor NaN
    ms, vs = (torch.exp2(torch.rand(n // 128 + 1, generator=gen) * 8 - 20) for _ in range(2))
    m[1280:1536], v[1280:1536] = 0, 0
    param = torch.randn(n, generator=gen).to(p)
    d = [x.to(DEV) for x in (param, grad, m, v, ms, vs)]
    norm, most = torch.tensor([3.7]), 0.8
    mxq.AdamW(*[[x] for x in d]).step(t, 1e-3, (b1, b2), seed=seed, norm=norm.to(DEV) if clip else None, max_norm=most)
    f = lambda x: torch.tensor(x, dtype=F32)
    spread32 = lambda s: s.repeat_interleave(128)[:n]
    x = grad.float()
    if clip:
        x = x * (f(1.0) / (norm + f(1e-6)) * f(most)).clamp(max=1.0)
    nm = f(b1) * (m.view(E4).float() * spread32(ms)) + f(1 - b1) * x
    nv = f(b2) * (v.view(E5).float() * spread32(vs)) + f(1 - b2) * x * x
    for new, codes, scale, kind, top in ((nm, d[2], d[4], E4, 448.0), (nv, d[3], d[5], E5, 57344.0)):
        most_of = torch.nn.functional.pad(new.abs(), (0, -n % 128)).view(-1, 128).amax(1)
        want = torch.maximum(most_of * (f(1.0) / f(top)), f(2.0 ** -120))
        assert torch.equal(scale.cpu(), want)
        y = (new / spread32(want)).clamp(-top, top)
        if kind is E4:
            want = y.to(E4)
        else:
            y = y.double()
            unit = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -14))) - 2)
            k = (torch.floor(y / unit + chance(0, n, t, seed).cpu().double() / 65536) * unit).clamp(max=top)
            want = torch.where((y > 0) & (k == 0), 2.0 ** -16, k).to(E5)
        off = codes.cpu() != want.view(U8)
        assert not bool(off.any()), (kind, int(off.sum()), off.nonzero()[:4, 0].tolist())


@pytest.mark.parametrize("eps,beta2", [(6e-11, 1 - 1e-7), (1e-10, 1 - 1e-8), (1e-8, 0.999), (1e-30, 0.999)])
def test_roots_of_subnormal_moments(eps, beta2):
    """v below binary32's least normal number, its root raised by 1 - beta2^t: it counts next to eps where it reaches its last
    places.  Gradients up to g with (1 - beta2) g^2 = 2^-126; the update's bound as test_gpu_adamw's, 30 half steps, and v's own
    rounding to a subnormal's step."""
    g = torch.logspace(-4, 0, 512, device=DEV) * (2.0 ** -63 / math.sqrt(1 - beta2) * 0.99)
    p, m, v = (torch.zeros(512, device=DEV) for _ in range(3))
    mxq.AdamW([p], [g], [m], [v]).step(1, 1.0, (0.0, beta2), eps, 0.0)
    g = g.double()
    exact = (1 - beta2) * g * g
    off = 8 * h * exact + 2.0 ** -149
    lo, hi = (g / (((exact + s * off).clamp(min=0.0) / (1 - beta2)).sqrt() + eps) for s in (1, -1))
    got = -p.double()
    assert bool(((got >= lo * (1 - 30 * h)) & (got <= hi * (1 + 30 * h))).all()), float(((got - lo) / lo).abs().max())
