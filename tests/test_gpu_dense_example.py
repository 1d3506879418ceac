"""The training example with AdamW: it runs, its gradients enter the update clipped, and the projection that the next step
takes is the rounded one of the parameters."""
import os
import sys

import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_a_run_with_adamw():
    require_gpu()
    from moe_train_step import Layer, train
    losses, layer = train(tokens=300, hidden=256, inter=128, experts=8, topk=2, vocab=1000, steps=3, rate=3e-3, adamw=True)
    assert all(x == x and abs(x) < 1e4 for x in losses)
    start = Layer(300, 256, 128, 8, 2, 1000)
    assert torch.equal(layer.proj, layer.proj_master.to(torch.bfloat16))
    assert torch.equal(layer.router, layer.router_master)
    for a, b in ((layer.router, start.router), (layer.proj_master, start.proj_master)):
        # every step moves an element by at most the rate times sqrt((1 - b1)^2 / (1 - b2)) and a little for decay
        moved = (a - b).abs()
        assert 0.0 < float(moved.max()) <= 3 * 3e-3 * 2.5 and float((moved > 0).float().mean()) > 0.5
