"""GPU tests of clipping where the norm, or its ratio to the limit, leaves
binary32's range or normal numbers.

Tolerance: out = in * min(1, max_norm / (norm + 1e-6)), all in binary64 (each
operation off by 2^-53, the squares' sum by their count times that), rounded
to binary32 and, for bf16, then to bf16: half a step of each, which is
2^-150 absolute where the result is subnormal in binary32 (2^-134 in bf16)."""
import math

import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from gpu_helpers import require_gpu
from test_gpu_train_ops import BF, F32, F64, H, HF, gen

pytestmark = pytest.mark.gpu
STEP = {F32: 2.0 ** -150, BF: 2.0 ** -134}  # half of the smallest


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("many", [False, True], ids=["few chunks", "many chunks"])
@pytest.mark.parametrize("size,max_norm", [(1e37, 1e-3), (3e38, 1e-3), (3e38, 1.0), (1e38, 1e-6), (3e-39, 1e-12), (1e36, 2.0),
                                           (1.0, 1.0), (1e-3, 0.5), (1e20, 1e-30)])
def test_clip_to_half_a_step(size, max_norm, many):
    g = gen(int(math.log2(size)) + 500)
    n = 4100 * 8192 if many else 5000
    host = [torch.randn(n, generator=g).clamp(-1, 1).to(BF), torch.randn(777, generator=g).clamp(-1, 1)]
    host = [(h.double() * size).to(h.dtype) for h in host]
    grads = [h.cuda() for h in host]
    out = [torch.full_like(d, 7.0) for d in grads]
    norm = torch.zeros(1, device="cuda")
    mxq.GradientSet(grads, out).clip(max_norm, norm)
    total = float(sum(h.double().square().sum() for h in host).sqrt())
    want_norm = torch.tensor([total], dtype=F64).to(F32)
    assert float(norm) == float(want_norm) or abs(float(norm) - total) <= 2 * HF * total
    limit = float(torch.tensor(max_norm, dtype=F32))
    coef = min(1.0, limit / (total + 1e-6))
    for h, o in zip(host, out):
        want = h.double() * coef
        half = HF * want.abs() + STEP[F32] + (H[BF] * want.abs() + STEP[BF] if h.dtype == BF else 0.0)
        err = (o.cpu().double() - want).abs()
        bad = err > (1 + 1e-6) * half
        assert not bool(bad.any()), f"{h.dtype}: off by {float((err / half).max()):.3g} half steps"
