"""8-bit moments with a value that is not finite: its block of 64 reads as NaN, whatever the value's kind,
and the other blocks keep their bits.  A finite gradient above 1.8e19 has such a square in float."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import optim as oo

from test_gpu_adamw import HYPER, Net

pytestmark = pytest.mark.gpu

AT = 70   # in tensor 7, whose second block it is


def quiet(net):
    """Gradients and moments of some neighbours are zero."""
    at = net.opt.offsets[7]
    net.g[7][64:68] = 0
    net.m[at + 64:at + 72] = 0
    net.v[at + 64:at + 72] = 0


def blocks(x):
    return x.view(-1, 64)


@pytest.mark.parametrize("dtype, master", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("bad", [1e25, -1e25, float("inf"), -float("inf")])
def test_a_second_moment_that_overflows_reads_as_nan(device, dtype, master, bad):
    import torch
    net, ref = Net(device, dtype, 8, master, seed=17), Net(device, dtype, 8, master, seed=17)
    for x in (net, ref):
        quiet(x)
    net.g[7][AT] = bad
    net.step(step=1)
    ref.step(step=1)
    hit = net.opt.offsets[7] // 64 + 1
    (m, v), (rm, rv) = net.moments(), ref.moments()
    assert torch.isnan(blocks(v)[hit]).all() and torch.isnan(net.scales[1, hit])
    assert not blocks(net.v)[hit].any()
    if np.isfinite(bad):   # the first moment holds it
        assert torch.isfinite(blocks(m)[hit]).all()
    else:
        assert torch.isnan(blocks(m)[hit]).all() and torch.isnan(net.scales[0, hit])
    others = torch.arange(net.opt.blocks, device=device) != hit
    assert torch.equal(blocks(m)[others], blocks(rm)[others]) and torch.equal(blocks(v)[others], blocks(rv)[others])
    # the next step shows it: every weight of the block, and no other
    net.g[7][AT] = 0
    net.step(step=2)
    weights = np.concatenate(net.weights())
    gone = np.isnan(weights)
    first = sum(net.opt.sizes[:7]) + 64
    assert gone[first:first + 64].all() and gone.sum() == 64


@pytest.mark.parametrize("max_norm", [0.0, 1.0])
def test_a_large_gradient_with_its_norm(device, max_norm):
    """The norm, in double, is finite: clipped by it, the square fits; without clipping the block reads as NaN."""
    import torch
    net = Net(device, "f32", 8, False, seed=18)
    quiet(net)
    net.g[7][AT] = 1e25
    norm = cg.grad_norm(net.opt, net.g)
    assert torch.isfinite(norm).all()
    net.step(step=1, norm=norm, max_norm=max_norm)
    hit = net.opt.offsets[7] // 64 + 1
    m, v = net.moments()
    if max_norm:
        assert torch.isfinite(m).all() and torch.isfinite(v).all()
    else:
        assert torch.isnan(blocks(v)[hit]).all() and int(torch.isnan(v).sum()) == 64
    # a norm that is not finite changes nothing
    net.g[7][AT] = float("inf")
    before = net.copies()
    net.step(step=2, norm=cg.grad_norm(net.opt, net.g), max_norm=max_norm)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, net.copies()))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_codes_written_from_values_that_are_not_finite(device, bad):
    """Codes and scales of the definition, every block's."""
    import torch
    opt, rng, f = cg.AdamW([640], "f32", 8), np.random.default_rng(19), np.float32
    m_in, v_in = np.zeros(opt.elements, f), np.zeros(opt.elements, f)
    m_in[:640], v_in[:640] = rng.standard_normal(640), np.exp(rng.standard_normal(640))
    v_in[130:140] = 0
    m_in[70], v_in[135] = -bad, bad
    m, v, scales, _ = opt.state(device)
    cg.adamw_state_write(opt, torch.from_numpy(m_in).to(device), torch.from_numpy(v_in).to(device), m, v, scales)
    cm, am = oo.codes(m_in, 127, True)
    cs, as_ = oo.codes(np.sqrt(v_in), 255, False)
    assert np.array_equal(m.cpu().numpy(), cm) and np.array_equal(v.cpu().numpy(), cs)
    assert np.array_equal(scales.cpu().numpy(), np.stack([am, as_]), equal_nan=True)
    a, b = cg.adamw_state_read(opt, m, v, scales)
    assert int(torch.isnan(a).sum()) == 64 and torch.isnan(blocks(a)[1]).all()
    assert int(torch.isnan(b).sum()) == 64 and torch.isnan(blocks(b)[2]).all()
