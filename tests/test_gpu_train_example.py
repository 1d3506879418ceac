"""The training example: its losses fall, and its gradients are those of the
same step in 64 bits."""
import os
import sys

import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_losses_fall():
    from moe_train_step import train
    losses, layer = train(tokens=300, hidden=256, inter=128, experts=8, topk=2, vocab=1000, steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert float(layer.norm) > 0.0


def test_router_gradient_of_the_step():
    """With the experts' rows as the layer computed them, the router's gradient from 64-bit autograd."""
    from moe_train_step import Layer
    T, C, E, k, V = 200, 256, 8, 2, 700
    layer = Layer(T, C, 128, E, k, V, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    h = torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    layer.forward(h, targets)
    layer.backward(h, targets)
    router = layer.router.double().requires_grad_()
    proj = layer.proj.double().requires_grad_()
    p = torch.softmax(h.double() @ router.t(), 1).gather(1, layer.ids.long())
    rows = layer.rows.double()[layer.pos.long()]
    y = ((p / p.sum(1, keepdim=True))[..., None] * rows).sum(1)
    loss = torch.nn.functional.cross_entropy((h.double() + y) @ proj.t(), targets)
    loss.backward()
    # x, dx and the projection's gradient are rounded to bf16 on the way: three half steps of 2^-8, norm against norm
    for got, want in ((layer.drouter, router.grad), (layer.dproj.double(), proj.grad)):
        assert float((got.double() - want).norm()) <= 3 * 2.0 ** -8 * float(want.norm())
