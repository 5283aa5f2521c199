"""The example with a mixture of experts behind its blocks: eager and captured steps alike, gradients by differences."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_captured_steps_are_the_eager_ones(device):
    import train_blocks
    a = train_blocks.train(steps=6, nodes=300, edges=3000, experts=4, graph=False)
    b = train_blocks.train(steps=6, nodes=300, edges=3000, experts=4)
    assert a == b and all(v == v for v in a)


def test_gradients_by_differences(device):
    import torch
    import train_blocks
    net, x, want = train_blocks.setup(nodes=60, edges=400, experts=3, dtype="f64")
    u, kept = net.forward(x)
    g = torch.randn(u.shape, dtype=u.dtype, device=device, generator=torch.Generator(device=device).manual_seed(1))
    net.backward(g, kept)
    gen = torch.Generator(device=device).manual_seed(2)
    h = 1e-6  # truncation h^2, cancellation 2^-53 / h of sums of some 1e3
    for i, (p, grad) in enumerate(zip(net.params, net.grads)):
        v = torch.randn(p.shape, generator=gen, device=device, dtype=p.dtype)
        keep, sides = p.clone(), []
        for s in (h, -h):
            p.copy_(keep + s * v)
            out, k = net.forward(x)
            assert k[-1][5].equal(kept[-1][5])  # the choice of experts stays: the differences are of one smooth piece
            sides.append((out * g).sum().item())
        p.copy_(keep)
        slope = (grad * v).sum().item()
        assert abs((sides[0] - sides[1]) / (2 * h) - slope) < 1e-5 * (1 + abs(slope)), i
