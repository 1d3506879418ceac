"""The AdamW step against its definition in 64 bits (GPU), moments in 32 bits and in 8.

Tolerances, h = 2^-24 (half a step of binary32, relative), counting the roundings:
  m        beta and 1 - beta as binary32, two products, the gradient's own (with a norm) and the sum: 6 h of the terms' magnitudes
  v        the same and one more product: 8 h
  update   m's; v's, halved by the root; the root, its scale, eps, their sum, the reciprocal (one step each at most: 2 h)
           and the two products: 16 h of the update
  param    the decay's product and the sum: 3 h of |param|; then its type's rounding
  codes    y = x / scale is off by 16 h of y; an E4M3 code by half a step more, an E5M2 code lies within a step
"""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64, U8 = "cuda", torch.bfloat16, torch.float32, torch.float64, torch.uint8
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
h = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: h}
SIZES = [1, 7, 8, 127, 128, 129, 1000, 2047, 8191, 8192, 8193, 20001, 0, 65536]


def rn(n, gen, std=1.0):
    return torch.randn(n, generator=gen, device=DEV) * std


def spread(scale, n):
    return scale.double().repeat_interleave(128)[:n]


def quantized(x, kind):
    n, top = x.numel(), 448.0 if kind is E4 else 57344.0
    s = (torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128).abs().amax(1) / top).clamp(min=2.0 ** -120)
    return (x / s.repeat_interleave(128)[:n]).clamp(-top, top).to(kind).view(U8), s


class Case:
    """Tensors of the given sizes; `shift` elements into their memory, so that they start off the 16-byte boundaries."""

    def __init__(self, sizes, p, g, eight, copies, shift=0, seed=0, grad_std=1e-3):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def at(x):
            room = torch.empty(x.numel() + shift + 16, dtype=x.dtype, device=DEV)
            room[shift:shift + x.numel()] = x
            return room[shift:shift + x.numel()]
        self.sizes, self.eight = sizes, eight
        self.params = [at(rn(n, gen, 0.02).to(p)) for n in sizes]
        self.grads = [at(rn(n, gen, grad_std).to(g)) for n in sizes]
        m, v = [rn(n, gen, 2e-4) for n in sizes], [rn(n, gen, 1e-3).square() + 1e-9 for n in sizes]
        if eight:
            pairs = [[quantized(x, kind) for x in xs] for xs, kind in ((m, E4), (v, E5))]
            (self.m, self.ms), (self.v, self.vs) = (([at(q) for q, _ in ps], [at(s) for _, s in ps]) for ps in pairs)
        else:
            self.m, self.v, self.ms, self.vs = [at(x) for x in m], [at(x) for x in v], None, None
        self.copies = [at(torch.zeros(n, dtype=BF, device=DEV)) for n in sizes] if copies else None
        self.decay = [k % 3 != 1 for k in range(len(sizes))]

    def set(self):
        return mxq.AdamW(self.params, self.grads, self.m, self.v, self.ms, self.vs, copies=self.copies, decay=self.decay)

    def state(self, k):
        """Tensor k in 64 bits: param, grad, m, v."""
        n = self.sizes[k]
        m, v = self.m[k], self.v[k]
        if self.eight:
            m, v = m.view(E4).double() * spread(self.ms[k], n), v.view(E5).double() * spread(self.vs[k], n)
        return [x.double().clone() for x in (self.params[k], self.grads[k], m, v)]


def chance(first, n, t, seed):
    """The 16 bits of each element, from the header's definition."""
    M = (1 << 64) - 1
    x = (seed + t * 0x9E3779B97F4A7C15) & M
    x = ((x ^ x >> 30) * 0xBF58476D1CE4E5B9) & M
    x = ((x ^ x >> 27) * 0x94D049BB133111EB) & M
    word = (x ^ x >> 31) & 0xFFFFFFFF
    P = first * 8192 + torch.arange(n, device=DEV)
    U = 0xFFFFFFFF
    r = (P >> 1) & U ^ word ^ ((P >> 33) * 0x9E3779B1 & U)
    r = ((r ^ r >> 16) * 0x85EBCA6B) & U
    r = ((r ^ r >> 13) * 0xC2B2AE35) & U
    r = r ^ r >> 16
    return torch.where(P % 2 == 0, r & 0xFFFF, r >> 16)


def near(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol + HALF[got.dtype] * want.abs() + 1e-44)
    assert not bool(bad.any()), (what, int(bad.sum()), got.numel(), float((off / (tol + 1e-44)).max()))


def check(c, before, t, rate, betas, eps, wd, coef=1.0, seed=0):
    first, wrong, total = 0, 0, 0
    for k, n in enumerate(c.sizes):
        p, g, m, v = before[k]
        g = g * coef
        b1, b2 = betas
        tm, tv = 6 * h * (b1 * m.abs() + (1 - b1) * g.abs()), 8 * h * (b2 * v + (1 - b2) * g * g)
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        den = (v / (1 - b2 ** t)).sqrt() + eps
        unit = rate / (1 - b1 ** t) / den
        up = unit * m
        want = p * (1 - (rate * wd if c.decay[k] else 0.0)) - up
        tol = 3 * h * p.abs() + 16 * h * up.abs() + unit * tm + up.abs() * torch.where(v > 0, tv / (2 * v), 0.0)
        near(c.params[k], want, tol, ("param", n))
        if c.copies is not None:
            near(c.copies[k], want, tol, ("copy", n))
        if not c.eight:
            near(c.m[k], m, tm, ("m", n))
            near(c.v[k], v, tv, ("v", n))
        elif n:
            for x, tx, codes, scale, kind, top, least, digits in ((m, tm, c.m[k].view(E4), c.ms[k], E4, 448.0, -6, 3),
                                                                  (v, tv, c.v[k].view(E5), c.vs[k], E5, 57344.0, -14, 2)):
                blocks = torch.nn.functional.pad(x.abs(), (0, -n % 128)).view(-1, 128).amax(1)
                ts = torch.nn.functional.pad(tx, (0, -n % 128)).view(-1, 128).amax(1) / top + 4 * h * blocks / top
                near(scale, (blocks / top).clamp(min=2.0 ** -120), ts, ("scale", n))
                s = spread(scale, n)
                y = (x / s).abs().clamp(max=top)
                err = tx / s + 16 * h * y
                step = torch.exp2(torch.floor(torch.log2((y + err).clamp(min=2.0 ** least))) - digits)
                code = codes.double()
                off = (code.abs() - y).abs()
                if kind is E4:
                    assert bool((off <= step / 2 + err).all()) and bool((code * x >= 0).all()), ("m", n)
                else:
                    assert bool((off <= step + err).all()) and bool((code > 0)[v > 0].all()), ("v", n)
                    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** least))) - digits)
                    expect = torch.floor(y / step + chance(first, n, t, seed).double() / 65536) * step
                    expect = torch.where((expect == 0) & (y > 0), 2.0 ** -16, expect.clamp(max=top))
                    wrong += int((expect != code).sum())
                    total += n
        first += -(-n // 8192)
    # the floor's argument is off by err / step, below 8 (8 + 16) h: that share of the codes may be one further
    assert wrong <= 3 + total * 8 * 24 * h * 3, (wrong, total)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("p,g", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
def test_step(p, g, eight, copies, shift):
    if copies and p is BF:
        pytest.skip("a copy is of float32 parameters")
    c = Case(SIZES, p, g, eight, copies, shift, seed=shift + 2 * eight)
    opt = c.set()
    for t, wd in ((1, 0.1), (2, 0.0), (700, 0.01)):
        before = [c.state(k) for k in range(len(SIZES))]
        opt.step(t, 3e-3, (0.9, 0.999), 1e-8, wd, seed=t * 77)
        check(c, before, t, 3e-3, (0.9, 0.999), 1e-8, wd, seed=t * 77)


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("norm", [0.25, 1.0, 40.0])
def test_gradients_are_clipped_on_the_way(eight, norm):
    c = Case([513, 9000], F32, BF, eight, True, seed=5, grad_std=norm / math.sqrt(9513))
    total = torch.empty(1, device=DEV)
    mxq.GradientSet(c.grads).norm(total)
    want = math.sqrt(sum(float(x.double().square().sum()) for x in c.grads))
    assert abs(float(total) - want) <= h * want * 1.01
    before = [c.state(k) for k in range(2)]
    c.set().step(10, 1e-3, (0.9, 0.95), norm=total, max_norm=0.5)
    check(c, before, 10, 1e-3, (0.9, 0.95), 1e-8, 0.01, coef=min(1.0, 0.5 / (float(total) + 1e-6)))


def test_the_norm_alone_is_clips_norm():
    gen = torch.Generator(device=DEV).manual_seed(1)
    for sizes in ([1], [3, 0, 100000], [8192 * 5000 + 3]):
        a, b = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        grads = [rn(n, gen).to(BF) for n in sizes]
        kept = [x.clone() for x in grads]
        mxq.GradientSet(grads).norm(a)
        assert all(torch.equal(x, y) for x, y in zip(grads, kept))
        mxq.GradientSet(grads).clip(1e30, b)
        assert torch.equal(a, b) and float(a) > 0


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
def test_a_captured_step_follows_rate_and_number(eight):
    c = Case([8192, 777], F32, F32, eight, False, seed=9)
    twin = Case([8192, 777], F32, F32, eight, False, seed=9)
    t, rate = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, device=DEV)
    opt, other = c.set(), twin.set()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(t, rate, seed=3)
    for k, r in ((1, 1e-3), (2, 5e-4), (3, 2.5e-4), (100, 1e-4)):
        t.fill_(k)
        rate.fill_(r)
        graph.replay()
        other.step(k, float(rate), seed=3)
        torch.cuda.synchronize()
        for a, b in zip(c.params + c.m + c.v, twin.params + twin.m + twin.v):
            assert torch.equal(a, b), (k, r)


def test_8bit_moments_of_zero_and_of_nothing_finite():
    n = 300
    z = lambda *s, dtype=U8: torch.zeros(*s, dtype=dtype, device=DEV)
    p, g = torch.ones(n, device=DEV), z(n, dtype=F32)
    m, v, ms, vs = z(n), z(n), z(3, dtype=F32), z(3, dtype=F32)
    opt = mxq.AdamW([p], [g], [m], [v], [ms], [vs])
    opt.step(1, 1e-3, weight_decay=0.0)  # no gradient, no moments: nothing moves
    assert torch.equal(p, torch.ones_like(p)) and not m.any() and not v.any()
    g[5], g[140], g[141] = 1.0, float("nan"), float("inf")
    opt.step(2, 1e-3, weight_decay=0.0)
    assert bool(m.view(E4).float()[140].isnan()) and bool(v.view(E5).float()[140].isnan()) and bool(p[140].isnan())
    assert float(m.view(E4).float()[141]) == 448.0 and float(v.view(E5).float()[141]) == 57344.0  # saturated
    ok = torch.ones(n, dtype=torch.bool, device=DEV)
    ok[[5, 140, 141]] = False
    assert torch.equal(p[ok], torch.ones_like(p[ok])) and bool(ms.isfinite().all()) and bool(vs.isfinite().all())
    assert float(p[5]) < 1.0 and not m[:5].any() and not m[150:].any()


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "8bit"])
@pytest.mark.parametrize("std", [1e-25, 1e-19, 1e-12, 1e12])
def test_gradients_of_any_size(std, eight):
    """Squares that are subnormal or vanish, and large ones."""
    c = Case([1111], F32, F32, eight, False, seed=3, grad_std=std)
    for xs in (c.m, c.v):
        xs[0].zero_()
    before = [c.state(0)]
    c.set().step(1, 1e-3, (0.9, 0.999), 1e-30)
    p, g, m, v = before[0]
    m, v = 0.1 * g, 0.001 * g * g
    # v itself is rounded to a subnormal's step
    tv = 8 * h * v + 2.0 ** -149
    lo, hi = ((x.clamp(min=0.0) / 0.001).sqrt() + 1e-30 for x in (v - tv, v + tv))
    a, b = (p * (1 - 1e-5) - 1e-3 / 0.1 * m / d for d in (lo, hi))
    tol = 3 * h * p.abs() + 30 * h * torch.maximum((p - a).abs(), (p - b).abs())
    got = c.params[0].double()
    assert bool(((got >= torch.minimum(a, b) - tol) & (got <= torch.maximum(a, b) + tol)).all())


def test_8bit_v_follows_a_gradient_that_shrinks():
    """The mean of sqrt(v) after the gradients of every second element shrank by 4: what rounding to nearest would lose."""
    n, gen = 1 << 15, torch.Generator(device=DEV).manual_seed(2)
    z = lambda k, dtype=U8: torch.zeros(k, dtype=dtype, device=DEV)
    p, g, m, v, ms, vs = z(n, F32), z(n, F32), z(n), z(n), z(n // 128, F32), z(n // 128, F32)
    exact = torch.zeros(n, dtype=F64, device=DEV)
    opt = mxq.AdamW([p], [g], [m], [v], [ms], [vs])
    for t in range(1, 801):
        g.copy_(rn(n, gen))
        if t > 200:
            g[::2] *= 0.25
        exact = 0.99 * exact + 0.01 * g.double() ** 2
        opt.step(t, 0.0, (0.9, 0.99), weight_decay=0.0, seed=1)
    ratio = (v.view(E5).double() * spread(vs, n) / exact).sqrt()
    # a code's own rounding is unbiased with a spread below 30%: the mean of 16384 is off by less than 2%, and by
    # E[sqrt] - sqrt(E), an eighth of the variance
    for part in (ratio[::2], ratio[1::2]):
        assert 0.95 < float(part.mean()) < 1.02, float(part.mean())


def test_two_runs_and_another_stream_give_the_same():
    runs = []
    for k in range(3):
        c = Case(SIZES, F32, BF, True, True, seed=4)
        opt = c.set()
        stream = torch.cuda.Stream() if k == 2 else torch.cuda.current_stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for t in range(1, 4):
                opt.step(t, 1e-2, seed=6)
        torch.cuda.synchronize()
        runs.append(c.params + c.m + c.v + c.ms + c.vs + c.copies)
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_what_lies_beside_the_tensors_stays():
    """Short tensors between guards, every alignment."""
    for eight in (False, True):
        for n in (1, 3, 9, 129):
            for shift in range(5):
                c = Case([n], F32, BF, eight, True, shift, seed=n)
                every = c.params + c.m + c.v + c.copies + (c.ms + c.vs if eight else [])
                rooms = [x._base for x in every]
                kept = [r.clone() for r in rooms]
                c.set().step(1, 1e-3)
                for x, r, k in zip(every, rooms, kept):
                    new, old = r.view(U8), k.view(U8)
                    a, b = shift * r.element_size(), (shift + x.numel()) * r.element_size()
                    assert torch.equal(new[:a], old[:a]) and torch.equal(new[b:], old[b:])
