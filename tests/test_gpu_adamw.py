"""AdamW over many tensors on the GPU: the weights and moments against the float64 formula within
counted roundings, the 8-bit codes against their float32 definition bit by bit; clipping, skipped
steps, tensors without gradients, layouts, streams and graphs."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import optim as oo

from block_cases import unit, work_unit

pytestmark = pytest.mark.gpu

SIZES = (1, 5, 0, 2047, 2048, 2049, 64, 10_007, 3)
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
KINDS = [("f32", 32, False), ("f64", 32, False), ("bf16", 32, False), ("f16", 32, False), ("bf16", 32, True),
         ("f32", 8, False), ("bf16", 8, True), ("f16", 8, False), ("f16", 8, True)]


class Net:
    """Tensors at odd elements of one buffer, their gradients, and moments with values."""

    def __init__(self, device, dtype, bits, master, sizes=SIZES, seed=0, shift=1):
        import torch
        self.opt = cg.AdamW(sizes, dtype, bits, master)
        o, rng = self.opt, np.random.default_rng(seed)
        total = sum(sizes) + len(sizes) * 3 + shift
        self.flat = torch.full((total,), 7.0, dtype=o.torch_dtype, device=device)
        gflat = torch.zeros(total, dtype=o.torch_dtype, device=device)
        self.p, self.g, at = [], [], shift
        for n in sizes:
            self.p.append(self.flat[at:at + n])
            self.g.append(gflat[at:at + n])
            self.p[-1].copy_(torch.from_numpy(rng.standard_normal(n)))
            self.g[-1].copy_(torch.from_numpy(rng.standard_normal(n) * np.exp(rng.standard_normal(n))))
            at += n + 3
        self.m, self.v, self.scales, self.master = o.state(device, self.p)
        m = np.zeros(o.elements)
        v = np.zeros(o.elements)
        for n, off in zip(sizes, o.offsets):
            m[off:off + n] = rng.standard_normal(n) * 0.3
            v[off:off + n] = np.exp(2 * rng.standard_normal(n))
        m, v = (torch.from_numpy(x).to(o.real_dtype).to(device) for x in (m, v))
        if bits == 8:
            cg.adamw_state_write(o, m, v, self.m, self.v, self.scales)
        else:
            self.m.copy_(m)
            self.v.copy_(v)
        if master:
            self.master += torch.from_numpy(rng.standard_normal(o.elements) * 1e-4).to(device) * (self.master != 0)

    def parts(self, flat):
        """A flat buffer's values, tensor by tensor, as numpy."""
        x = flat.cpu().numpy()
        return [x[o:o + n] for n, o in zip(self.opt.sizes, self.opt.offsets)]

    def moments(self):
        if self.opt.state_bits == 8:
            return cg.adamw_state_read(self.opt, self.m, self.v, self.scales)
        return self.m.clone(), self.v.clone()

    def weights(self):
        if self.master is not None:
            return [x.astype(np.float64) for x in self.parts(self.master)]
        return [t.double().cpu().numpy() for t in self.p]

    def step(self, **kw):
        cg.adamw_step(self.opt, self.p, self.g, self.m, self.v, self.scales, self.master, **{**HYPER, **kw})

    def copies(self):
        return [t.clone() for t in (self.flat, self.m, self.v, self.scales, self.master) if t is not None]


def check_step(net, dtype, want_p, want_m, want_v, before, factor=1.0):
    """m, v: three roundings of each of two terms, the scalars' and the gradient's scaling; p: those
    through the quotient, and a step's own."""
    w = work_unit(dtype)
    m, v = net.moments()
    got_p = net.weights()
    for i in range(len(want_p)):
        m0, v0, p0, g = before[0][i], before[1][i], before[2][i], before[3][i] * factor
        msize = HYPER["beta1"] * np.abs(m0) + (1 - HYPER["beta1"]) * np.abs(g)
        if net.opt.state_bits == 32:
            assert np.all(np.abs(net.parts(m)[i] - want_m[i]) <= 6 * w * msize)
            assert np.all(np.abs(net.parts(v)[i] - want_v[i]) <= 8 * w * want_v[i])
        t = before[4]
        mhat = msize / (1 - HYPER["beta1"] ** t)
        move = HYPER["lr"] * mhat / (np.sqrt(want_v[i] / (1 - HYPER["beta2"] ** t)) + HYPER["eps"])
        most = 3 * w * np.abs(p0) + 24 * w * move
        if net.master is None:
            most = most + (unit(dtype) * np.abs(want_p[i]) + (2.0 ** -25 if dtype == "f16" else 0)
                           if dtype in ("bf16", "f16") else 0)
        assert np.all(np.abs(got_p[i] - want_p[i]) <= most), (i, np.max(np.abs(got_p[i] - want_p[i]) / most))


def expected(net, t, factor=1.0):
    m, v = net.moments()
    before = ([x.astype(np.float64) for x in net.parts(m)], [x.astype(np.float64) for x in net.parts(v)],
              net.weights(), [g.double().cpu().numpy() for g in net.g], t)
    res = [oo.adamw(p, g, a, b, step=t, factor=factor, **HYPER) for a, b, p, g in zip(*before[:4])]
    return [list(x) for x in zip(*res)], before


@pytest.mark.parametrize("dtype, bits, master", KINDS)
def test_steps_against_the_formula(device, dtype, bits, master):
    import torch
    net = Net(device, dtype, bits, master)
    edges = net.flat.clone()
    for t in (1, 2, 500):
        (p, m, v), before = expected(net, t)
        net.step(step=t)
        check_step(net, dtype, p, m, v, before)
        if master:
            for x, y in zip(net.p, net.parts(net.master)):
                assert torch.equal(x.cpu(), torch.from_numpy(y).to(net.opt.torch_dtype))
    # between the tensors nothing is written, and the moments' padding stays zero
    inside = torch.zeros_like(net.flat, dtype=torch.bool)
    for t in net.p:
        inside[t.storage_offset():t.storage_offset() + t.numel()] = True
    assert torch.equal(net.flat[~inside], edges[~inside])
    pad = torch.ones(net.opt.elements, dtype=torch.bool, device=device)
    for n, off in zip(net.opt.sizes, net.opt.offsets):
        pad[off:off + n] = False
    for s in (net.m, net.v, net.master):
        assert s is None or not s[pad].any()


@pytest.mark.parametrize("dtype, master", [("f32", False), ("bf16", True), ("f16", False)])
def test_codes_are_those_of_the_definition(device, dtype, master):
    """The moments' arithmetic in float32, rounding by rounding, and the codes from it: equal bits."""
    net = Net(device, dtype, 8, master, seed=3)
    f = np.float32
    for t in (1, 2, 3):
        m, v = (x.cpu().numpy() for x in net.moments())
        g = np.zeros(net.opt.elements, f)
        for n, off, gi in zip(net.opt.sizes, net.opt.offsets, net.g):
            g[off:off + n] = gi.float().cpu().numpy()
        m = m * f(HYPER["beta1"]) + g * f(1 - HYPER["beta1"])
        v = v * f(HYPER["beta2"]) + g * g * f(1 - HYPER["beta2"])
        net.step(step=t)
        cm, am = oo.codes(m, 127, True)
        cs, as_ = oo.codes(np.sqrt(v), 255, False)
        assert np.array_equal(net.m.cpu().numpy(), cm) and np.array_equal(net.v.cpu().numpy(), cs)
        assert np.array_equal(net.scales.cpu().numpy(), np.stack([am, as_]))
        got = net.moments()
        assert np.array_equal(got[0].cpu().numpy(), oo.values(cm, am, 127).reshape(-1))
        assert np.array_equal(got[1].cpu().numpy(), np.square(oo.values(cs, as_, 255).reshape(-1)))


def test_codes_decay_when_gradients_cease(device):
    """A block's second moment follows its decay although each step moves it by far less than a code."""
    net = Net(device, "f32", 8, False, sizes=(640,), seed=4)
    before = net.moments()[1][:640].double()
    net.g[0].zero_()
    for t in range(1, 201):
        net.step(step=t)
    after = net.moments()[1][:640].double()
    want = HYPER["beta2"] ** 200
    ratio = after.view(-1, 64).amax(1) / before.view(-1, 64).amax(1)
    assert abs(ratio / want - 1).max().item() < 200 * 8 * 2.0 ** -24  # the largest of a block carries no code's error
    assert (after > 0).all()


@pytest.mark.parametrize("dtype, bits, master", [("f32", 32, False), ("bf16", 32, True), ("f32", 8, False)])
def test_norm_and_clipping(device, dtype, bits, master):
    net = Net(device, dtype, bits, master, seed=5)
    norm = cg.grad_norm(net.opt, net.g)
    want = np.sqrt(sum(np.square(g.double().cpu().numpy()).sum() for g in net.g))
    # squares of 32-bit values are exact in 64; every sum rounds once
    assert abs(norm.item() / want - 1) <= sum(SIZES) * 2.0 ** -53
    for max_norm, scale in ((0.5 * want, 1.0), (2 * want, 1.0), (0.1, -0.25), (0.0, 0.125)):
        factor = oo.clip_factor(want, max_norm, scale)
        (p, m, v), before = expected(net, 7, factor)
        net.step(step=7, norm=norm, max_norm=max_norm, grad_scale=scale)
        check_step(net, dtype, p, m, v, before, factor)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_step_whose_norm_is_not_finite_changes_nothing(device, bad):
    import torch
    for dtype, bits, master in (("f32", 32, False), ("bf16", 8, True)):
        net = Net(device, dtype, bits, master, seed=6)
        net.g[7][5000] = bad
        norm = cg.grad_norm(net.opt, net.g)
        assert not torch.isfinite(norm).any()
        before = net.copies()
        net.step(step=1, norm=norm, max_norm=1.0)
        net.step(step=1, norm=norm)
        assert all(torch.equal(a, b) for a, b in zip(before, net.copies()))


def test_a_gradient_that_is_not_finite_stays_in_its_block(device):
    import torch
    net, ref = Net(device, "f32", 8, False, seed=7), Net(device, "f32", 8, False, seed=7)
    net.g[7][70] = float("nan")
    net.step(step=1)
    ref.step(step=1)
    at = net.opt.offsets[7]
    a, b = net.moments(), ref.moments()
    for x, y in zip(a, b):
        x, y = x.view(-1, 64), y.view(-1, 64)
        assert torch.isnan(x[at // 64 + 1]).all()
        x[at // 64 + 1] = y[at // 64 + 1]
        assert torch.equal(x, y)
    x, y = net.p[7].clone(), ref.p[7].clone()
    assert torch.isnan(x[70])
    x[70] = y[70]
    assert torch.equal(x, y)


def test_tensors_without_gradients_are_left_alone(device):
    import torch
    net = Net(device, "f32", 32, False, seed=8)
    before = net.copies()
    gone = (0, 3, 7)
    grads = [None if i in gone else g for i, g in enumerate(net.g)]
    norm = cg.grad_norm(net.opt, grads)
    want = np.sqrt(sum(np.square(g.double().cpu().numpy()).sum() for g in grads if g is not None))
    assert abs(norm.item() / want - 1) <= 1e-12
    cg.adamw_step(net.opt, net.p, grads, net.m, net.v, step=1, **HYPER)
    full = Net(device, "f32", 32, False, seed=8)
    full.step(step=1)
    for i, (n, off) in enumerate(zip(net.opt.sizes, net.opt.offsets)):
        for a, old, new in ((net.m, before[1], full.m), (net.v, before[2], full.v)):
            assert torch.equal(a[off:off + n], (old if i in gone else new)[off:off + n])
        if n and i not in gone:
            assert torch.equal(net.p[i], full.p[i])
    x = net.flat.clone()
    for i in gone:
        s = net.p[i].storage_offset()
        assert torch.equal(x[s:s + net.p[i].numel()], before[0][s:s + net.p[i].numel()])
    # none at all
    before = net.copies()
    cg.adamw_step(net.opt, net.p, [None] * len(SIZES), net.m, net.v, step=2, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(before, net.copies()))


@pytest.mark.parametrize("count", [1, 111, 112, 113, 300])
def test_more_tensors_than_a_launch_takes(device, count):
    rng = np.random.default_rng(count)
    sizes = tuple(int(n) for n in rng.integers(0, 5000, count))
    net = Net(device, "f32", 32, False, sizes=sizes, seed=9)
    want = np.sqrt(sum(np.square(g.double().cpu().numpy()).sum() for g in net.g))
    assert abs(cg.grad_norm(net.opt, net.g).item() / want - 1) <= 1e-11
    (p, m, v), before = expected(net, 3)
    net.step(step=3)
    check_step(net, "f32", p, m, v, before)


def test_large_tensor(device):
    """More units than the norm has workgroups, in one tensor, against torch in double on the GPU."""
    import torch
    n = 2048 * 2048 * 3 + 77
    gen = torch.Generator(device=device).manual_seed(1)
    p = torch.randn(n, generator=gen, device=device)
    g = torch.randn(n, generator=gen, device=device)
    opt = cg.AdamW([n])
    m, v, _, _ = opt.state(device)
    norm = cg.grad_norm(opt, [g])
    assert abs(norm.item() / g.double().norm().item() - 1) < 1e-12
    want = p.double()
    cg.adamw_step(opt, [p], [g], m, v, step=1, **HYPER)
    gd = g.double()
    want = want * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * gd / (gd.abs() + HYPER["eps"])
    assert ((p.double() - want).abs() <= 2.0 ** -24 * (3 * want.abs() + 24 * HYPER["lr"]) + 2.0 ** -24 * 3e-3).all()
    assert not m[n:].any() and not v[n:].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_two_to_the_31(device, bits):
    """Offsets of 64 bits: the last units of a tensor of 2.2e9 elements step as a tensor of their own does."""
    import torch
    n, tail = (1 << 31) + 2048 * 7 + 5, 2048 * 9 + 5
    gen = torch.Generator(device=device).manual_seed(3)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=device) for _ in range(2))
    for t in (p, g):
        t[-tail:] = torch.randn(tail, generator=gen, device=device).to(torch.bfloat16)
    ps, gs = p[-tail:].clone(), g[-tail:].clone()
    for q, h, size in ((p, g, n), (ps, gs, tail)):
        opt = cg.AdamW([size], "bf16", bits)
        m, v, scales, _ = opt.state(device)
        norm = cg.grad_norm(opt, [h])
        for step in (1, 2):
            cg.adamw_step(opt, [q], [h], m, v, scales, step=step, norm=norm, max_norm=0.5, **HYPER)
        last = opt.elements - (tail + 2048 - 5)
        if size == n:
            kept = (norm, m[last:].clone(), v[last:].clone())
        else:
            assert abs(norm.item() / kept[0].item() - 1) < 1e-12
            assert torch.equal(m[last:], kept[1]) and torch.equal(v[last:], kept[2])
        del m, v, scales
    assert torch.equal(p[-tail:], ps) and not p[:-tail].any()


def test_state_round_trip(device):
    import torch
    net = Net(device, "f32", 8, False, seed=11)
    m, v = net.moments()
    m2, v2, s2 = torch.empty_like(net.m), torch.empty_like(net.v), torch.empty_like(net.scales)
    cg.adamw_state_write(net.opt, m, v, m2, v2, s2)
    a, b = cg.adamw_state_read(net.opt, m2, v2, s2)
    # decoded values are codes again: the same ones, up to the last bits of a root
    assert torch.equal(m2, net.m) and torch.equal(v2, net.v)
    assert torch.allclose(a, m, rtol=1e-6, atol=0) and torch.allclose(b, v, rtol=1e-6, atol=0)


def test_tensor_lists_follow_their_tensors(device):
    import torch
    net = Net(device, "f32", 32, False, sizes=(100, 50), seed=12)
    params, grads = cg.tensor_list(net.opt, net.p), cg.tensor_list(net.opt, net.g)
    net.g[0].data = torch.ones(100, device=device)   # elsewhere now
    cg.adamw_step(net.opt, params, grads, net.m, net.v, step=1, **HYPER)
    ref = Net(device, "f32", 32, False, sizes=(100, 50), seed=12)
    ref.g[0].fill_(1.0)
    ref.step(step=1)
    assert torch.equal(net.p[0], ref.p[0]) and torch.equal(net.m, ref.m)
    net.g[1].data = torch.ones(20, device=device)
    with pytest.raises(ValueError, match="20 elements"):
        cg.adamw_step(net.opt, params, grads, net.m, net.v, step=2, **HYPER)
    with pytest.raises(ValueError, match="another layout"):
        cg.grad_norm(cg.AdamW([100, 50]), grads)
    with pytest.raises(ValueError, match="contiguous"):
        cg.tensor_list(net.opt, [torch.zeros(200, device=device)[::2], net.p[1]])
    with pytest.raises(TypeError):
        cg.tensor_list(net.opt, [torch.zeros(100, device=device, dtype=torch.float64), net.p[1]])


@pytest.mark.parametrize("bits", [32, 8])
def test_schedule_streams_and_graph(device, bits):
    """Steps by a device schedule: the bits of steps by number; on a side stream; and replayed from a
    graph, with eager work and synchronizations between the replays."""
    import torch
    net, ref = (Net(device, "f32", bits, False, seed=13) for _ in range(2))
    sch = torch.tensor([0.0, HYPER["lr"], 0.0, 0.0], dtype=torch.float64, device=device)
    norm = torch.empty(1, dtype=torch.float64, device=device)
    ws = torch.empty(net.opt.norm_workspace, dtype=torch.uint8, device=device)
    params, grads = cg.tensor_list(net.opt, net.p), cg.tensor_list(net.opt, net.g)

    def step():
        cg.adamw_schedule(sch, HYPER["beta1"], HYPER["beta2"])
        cg.grad_norm(net.opt, grads, norm=norm, workspace=ws)
        cg.adamw_step(net.opt, params, grads, net.m, net.v, net.scales, schedule=sch, norm=norm, max_norm=3.0,
                      **{k: v for k, v in HYPER.items() if k != "lr"})

    def same(t):
        ref.step(step=t, norm=cg.grad_norm(ref.opt, ref.g), max_norm=3.0)
        torch.cuda.synchronize()
        # beta^t of the device and of the host may differ in the last bit of 64
        assert torch.equal(net.m, ref.m) and torch.equal(net.v, ref.v)
        assert torch.allclose(net.flat, ref.flat, rtol=2.0 ** -22, atol=1e-9)
        ref.flat.copy_(net.flat)
    step()
    same(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    same(2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (3, 4, 5):
        for a, b in zip(net.g, ref.g):
            a.copy_(torch.randn(a.shape, device=device))
            b.copy_(a)
        torch.cuda.synchronize()
        graph.replay()
        same(t)
        assert sch[0].item() == t
