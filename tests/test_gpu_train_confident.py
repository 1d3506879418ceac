"""GPU tests of the vocabulary cross entropy where one word is all but certain:
its loss is not negative, and no gradient has the wrong sign.

The definition: loss = log sum exp(z) - z_target >= 0 and p <= 1, whatever the
logits' magnitude.  Both hold for the rounded values too when the largest
logit's term of the sum is exactly one (rounding keeps the order: the sum is
then at least 1, its log at least 0, and lse at least the largest logit).
"""
import pytest
import torch

import mxfp4_precision_numerics_amd as mxq
from gpu_helpers import require_gpu
from test_gpu_train_ops import BF, HF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def confident(T, Hd, V, high):
    """Token t's logits are 0 but for those of its column's words, its target's among them: exact products of two 8-bit
    numbers, in (0, 2 high]."""
    t = torch.arange(T) * 7919 % V
    col = torch.arange(T) % Hd
    x, w = torch.zeros(T, Hd), torch.zeros(V, Hd)
    x[torch.arange(T), col] = torch.linspace(high / T, high, T, dtype=torch.float64).float()
    w[t, col] = 1.0 + (t * 37 % 128) / 128.0
    x, w = x.to(BF), w.to(BF)
    return x, w, t, col, x.double() @ w.double().t()


@pytest.mark.parametrize("T,Hd,V,high", [(37, 64, 1, 300.0), (300, 512, 300, 200.0), (500, 512, 1000, 1.0),
                                         (300, 512, 700, 20000.0), (200, 256, 500, 1e12), (1000, 1024, 4001, 200.0),
                                         (1500, 2048, 3000, 400.0), (4096, 512, 4096, 100.0)])
def test_a_loss_is_not_negative(T, Hd, V, high):
    x, w, t, col, z = confident(T, Hd, V, high)
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    ws = torch.full((mxq.linear_cross_entropy_workspace(T, Hd, V, True),), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = (torch.full((T,), 9.0, device="cuda") for _ in range(2))
    mxq.linear_cross_entropy(xd, wd, td, loss, lse, ws)
    top = z.amax(1).float().cuda()  # exact: products of two 8-bit numbers
    below = float((top - lse).max())
    assert below <= 0, "lse below the largest logit"
    mine = z.gather(1, t[:, None])[:, 0].float().cuda()
    least = float(loss.min())
    assert least >= 0, "a negative loss"
    # loss: lse's half step and the subtraction's, the sum of V terms, the log; the fast exponential of each term but the
    # largest, with its argument's size
    want = torch.logsumexp(z, 1)
    spread = z.amax(1) - z.amin(1)
    bound = 2 * HF * want.abs() + HF * ((V + 16) + 4 * (2 + spread) * (1 - (z.amax(1) - want).exp()))
    err = (loss.cpu().double() - (want - mine.cpu().double())).abs()
    assert bool((err <= bound).all()), f"off by {float((err / bound).max()):.3g} times the bound"
    # (p - 1) dloss of the target's word: never positive where dloss is 1
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    mxq.linear_cross_entropy_backward(xd, wd, td, lse, torch.ones(T, device="cuda"), dx, dw, ws)
    only = ((w != 0).sum(0) == 1)[col]  # the one word of the token's column: dx there is its g times a positive weight
    assert bool((dx[torch.arange(T), col].cpu()[only] <= 0).all()), "dx of a certain word has the wrong sign"
    own = ((x != 0).sum(0) == 1)[col]  # the one token of its column: dw there is its g times a positive entry of x
    assert bool((dw[t.cuda(), col.cuda()].cpu()[own] <= 0).all()), "dw of a certain word has the wrong sign"
    assert int(only.sum()) + int(own.sum()) > 0 or T > Hd
