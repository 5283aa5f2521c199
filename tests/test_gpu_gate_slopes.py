"""Gradients through gates far from 0, relative to their own size: open gates (large logits) keep their
slope as closed ones do."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import block as ob

from block_cases import DTYPES, unit, work_unit

pytestmark = pytest.mark.gpu

LOGITS = (-20.0, -12.0, -6.0, -3.0, 3.0, 6.0, 12.0, 20.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["sigmoid", "silu", "tanh"])
@pytest.mark.parametrize("gate", ["channel", "row"])
def test_slopes_of_open_and_closed_gates(device, gate, act, dtype):
    """grad_gate = act'(g) scale sum(grad_h f) with positive terms, so nothing cancels but the slope's own
    terms.  Counted: the exponential (1 step, so 2 halves), its sum, quotient and up to six products; the
    terms' products and the sum over 8 columns: 3 + 3; SiLU's 1 + g (1 - s), whose terms are at most 2.1 times
    their sum at these logits, doubles the slope's; under 32 in all.  The oracle's own in 64 bits: 32 more.  The 16-bit
    rows' hardware exponential is off by |x| 2^-23 and its argument x is g, or 2 g for tanh, and enters the
    slope up to twice (numerator and sum): 8 |g| of 2^-24, and its own and the reciprocal's last step, 8."""
    import torch
    d, rng = 8, np.random.default_rng(5)
    block = cg.block_for(f"{d}x0e", dtype, gate=gate, act=act)
    t, real = block.torch_dtype, block.real_dtype
    rows = len(LOGITS) * 5
    held = lambda a, ty: torch.from_numpy(np.ascontiguousarray(a)).to(ty)  # noqa: E731
    g = held(np.repeat(np.array(LOGITS), 5)[:, None] + np.zeros((rows, d if gate == "channel" else 1)), t)
    f, dh = (held(1 + rng.random((rows, d)), t) for _ in range(2))
    scale = held(1 + rng.random(d), real)
    got = cg.join_backward(block, dh.to(device), None, None, f.to(device), g.to(device), None, scale.to(device), None, None,
                           None)[2].double().cpu().numpy()
    n = [x.double().numpy() for x in (dh, f, g, scale)]
    want = ob.act(act, n[2])[1] * (n[0] * n[1] * n[3] if gate == "channel" else
                                   (n[0] * n[1] * n[3]).sum(1, keepdims=True))
    roundings = 64 + (8 + 8 * np.abs(n[2]) if dtype in ("bf16", "f16") else 0)
    most = (unit(dtype) + roundings * work_unit(dtype)) * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)
    off = np.abs(got - want) / most
    assert np.all(off <= 1), [(float(x), float(o)) for x, o in zip(n[2][:, 0], off.max(1)) if o > 1]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["sigmoid", "silu", "tanh"])
def test_gates_that_overflow_the_exponential(device, act, dtype):
    """At the ends of a 16-bit range and beyond the exponential's: slopes of 0 or 1, no NaN."""
    import torch
    block = cg.block_for("4x0e", dtype, gate="channel", act=act)
    ends = [-6e4, -800.0, -100.0, 100.0, 800.0, 6e4]
    g = torch.tensor(ends, dtype=block.torch_dtype, device=device)[:, None].expand(-1, 4).contiguous()
    one = torch.ones_like(g)
    out = cg.join_backward(block, one, None, None, one, g, None, None, None, None, None)
    want = [0.0, 0.0, 0.0] + ([1.0] * 3 if act == "silu" else [0.0] * 3)
    assert torch.allclose(out[2].double().cpu(), torch.tensor(want, dtype=torch.float64)[:, None].expand(-1, 4), rtol=0,
                          atol=1e-30)
    h = cg.join_forward(block, torch.zeros_like(g), one, g, None, None, None)[0]
    assert torch.isfinite(h).all()
