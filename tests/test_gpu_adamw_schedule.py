"""A device schedule with steps that are skipped: they are not counted, eagerly and in a captured graph."""
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg

from test_gpu_adamw import HYPER, Net

pytestmark = pytest.mark.gpu

BETAS = HYPER["beta1"], HYPER["beta2"]
REST = {k: v for k, v in HYPER.items() if k != "lr"}


def schedule(device):
    import torch
    return torch.tensor([0.0, HYPER["lr"], 0.0, 0.0], dtype=torch.float64, device=device)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_the_schedule_stays_where_the_norm_is_not_finite(device, bad):
    import torch
    sch, norm = schedule(device), torch.empty(1, dtype=torch.float64, device=device)
    for value, scale, step in ((2.0, 1.0, 1), (bad, 1.0, 1), (1e300, 1e10, 1), (bad, 0.0, 1), (0.0, -3.0, 2)):
        before = sch.clone()
        norm.fill_(value)
        cg.adamw_schedule(sch, *BETAS, norm=norm, grad_scale=scale)
        assert sch[0].item() == step
        if step == before[0].item():
            assert torch.equal(sch, before)
    want = schedule(device)
    for _ in range(2):
        cg.adamw_schedule(want, *BETAS)
    assert torch.equal(sch, want)


@pytest.mark.parametrize("dtype, bits, master", [("f32", 32, False), ("bf16", 32, True), ("f16", 8, True)])
def test_a_step_after_skipped_ones_is_the_step_alone(device, dtype, bits, master):
    """Captured: ten steps whose gradients overflow, good ones between and after them; the other network
    sees the good ones only, one by one.  Equal bits."""
    import torch
    net, ref = (Net(device, dtype, bits, master, seed=23) for _ in range(2))
    sch, rsch = schedule(device), schedule(device)
    norm = torch.empty(1, dtype=torch.float64, device=device)
    ws = torch.empty(net.opt.norm_workspace, dtype=torch.uint8, device=device)

    def step(x, s):
        cg.grad_norm(x.opt, x.g, norm=norm, workspace=ws)
        cg.adamw_schedule(s, *BETAS, norm=norm, grad_scale=0.5)
        cg.adamw_step(x.opt, x.p, x.g, x.m, x.v, x.scales, x.master, schedule=s, norm=norm, max_norm=3.0, grad_scale=0.5,
                      **REST)
    good = [g.clone() for g in net.g]
    net.g[7][100] = float("inf")
    before = net.copies()
    step(net, sch)   # eager: it changes nothing
    assert all(torch.equal(a, b) for a, b in zip(before, net.copies())) and sch[0].item() == 0
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(net, sch)
    taken = 0
    for fine in [False] * 4 + [True] + [False] * 6 + [True, True]:
        for a, b, c in zip(net.g, good, ref.g):
            a.copy_(b)
            c.copy_(b)
        if not fine:
            net.g[7][100] = float("nan")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if fine:
            taken += 1
            step(ref, rsch)
        assert sch[0].item() == taken and torch.equal(sch, rsch)
        assert all(torch.equal(a, b) for a, b in zip(net.copies(), ref.copies()))
