"""The training example: its gradients against differences of its loss, a loss that falls, and the
captured step against the eager one."""
import os
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if os.path.join(ROOT, "examples") not in sys.path:
    sys.path.append(os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_against_differences_of_the_loss(device):
    """Along a random direction of all weights.  float32 losses: the difference's rounding is about
    1e-6 of the loss over the step, its curvature the square of the step."""
    import torch
    import train_blocks as ex
    net, x, want = ex.setup(device, nodes=200, edges=3001)
    u, kept = net.forward(x)
    net.backward((u - want) * (2.0 / u.numel()), kept)
    gen = torch.Generator(device=device).manual_seed(7)
    way = [torch.randn(p.shape, generator=gen, device=device) * p.abs().mean() for p in net.params]
    ana = sum((g.double() * w.double()).sum().item() for g, w in zip(net.grads, way))
    start = [p.clone() for p in net.params]

    def loss(s):
        for p, a, w in zip(net.params, start, way):
            p.copy_(a + s * w)
        return (net.forward(x)[0].double() - want.double()).square().mean().item()
    step = 5e-3
    num = (8 * (loss(step) - loss(-step)) - (loss(2 * step) - loss(-2 * step))) / (12 * step)
    assert abs(num - ana) <= 5e-3 * abs(ana) + 1e-4, (num, ana)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_loss_falls_and_the_captured_step_is_the_eager_one(device, bits):
    import train_blocks as ex
    captured = ex.train(steps=25, bits=bits, device=device, nodes=500, edges=8000)
    eager = ex.train(steps=25, bits=bits, graph=False, device=device, nodes=500, edges=8000)
    assert np.array_equal(captured, eager)   # every kernel of the step is deterministic
    assert captured[-1] < 0.6 * captured[0] and np.all(np.isfinite(captured))
