"""Group norm over graphs on the GPU against the float64 oracle, element by element, within bounds that
count roundings (expert_cases); its edges, layouts, streams and graphs."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import experts as ox

from block_cases import work_unit
from expert_cases import (DTYPES, NORM_SHAPES, act_error, held, host, norm_inputs, norm_roundings, real, stat_bounds,
                          within)

pytestmark = pytest.mark.gpu

EPS = 1e-5


def up(a, device):
    import torch
    return (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(device)


def check_forward(norm, t, got, dtype, act, rows=None):
    y, mean, rstd = got
    x, w, bias, ptr = host(t["x"]), host(t["w"]), host(t["bias"]), t["ptr"]
    u, c = work_unit(dtype), norm_roundings(norm, rows or len(x))
    m, r = ox.group_stats(x, ptr, norm.groups, EPS)
    dm, dr = stat_bounds(x, ptr, m, r, u, c)
    within("mean", mean, m, dm)
    within("rstd", rstd, r, dr)
    # y from the statistics that were stored
    m, r = host(mean), host(rstd)
    want, z = ox.group_norm(x, ptr, w, bias, m, r, act)
    n, ch = x.shape
    xh = (x - ox.per_row(m, ptr, n, ch)) * ox.per_row(r, ptr, n, ch)
    dz = 5 * u * np.abs(xh * w) + 2 * u * (np.abs(xh * w) + np.abs(bias))
    inside = np.zeros((n, 1))
    inside[ptr[0]:ptr[-1]] = 1
    within("y", y, want, act_error(z, dz, u) * inside, dtype)


def check_backward(norm, t, mean, rstd, got, dtype, act, rows=None):
    x, w, bias, dy, ptr = host(t["x"]), host(t["w"]), host(t["bias"]), host(t["dy"]), t["ptr"]
    u, c = work_unit(dtype), norm_roundings(norm, rows or len(x)) + len(x)
    f = ox.group_norm_grad(x, ptr, w, bias, host(mean), host(rstd), dy, act)
    xh, z, q, r, means = f["xh"], f["z"], f["q"], f["r"], f["means"]
    inside = f["inside"]
    dslope = act_error(z, 4 * u * np.abs(xh * w) + 2 * u * (np.abs(xh * w) + np.abs(bias)), u)
    ddz = (np.abs(dy) * dslope + 2 * u * np.abs(f["dz"])) * inside
    dq = ddz * np.abs(w) + u * np.abs(q)
    dxh = 3 * u * np.abs(xh)
    mq = means(dq) + c * u * means(np.abs(q))
    mx = means(dq * np.abs(xh) + np.abs(q) * dxh) + c * u * means(np.abs(q * xh))
    most = np.abs(r) * (dq + mq + np.abs(xh) * mx + dxh * np.abs(means(q * xh)) +
                        6 * u * (np.abs(q) + np.abs(means(q)) + np.abs(xh * means(q * xh))))
    gx, gw, gb = got
    within("grad_x", gx, f["grad_x"] * inside, most * inside, dtype)
    within("grad_w", gw, f["grad_w"], (ddz * np.abs(xh) + np.abs(f["dz"]) * dxh + c * u * np.abs(f["dz"] * xh)).sum(0) + u * np.abs(f["grad_w"]))
    within("grad_bias", gb, f["grad_bias"], (ddz + c * u * np.abs(f["dz"])).sum(0) + u * np.abs(f["grad_bias"]))


def both(norm, t, device, **kw):
    d = {k: up(v, device) for k, v in t.items()}
    fwd = cg.group_norm_forward(norm, d["x"], d["ptr"], d["w"], d["bias"])
    bwd = cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], fwd[1], fwd[2], d["dy"])
    return fwd, bwd


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels, groups, graphs", NORM_SHAPES, ids=lambda v: str(len(v)) if isinstance(v, list) else str(v))
def test_shapes(device, channels, groups, graphs, dtype):
    norm = cg.group_norm_for(channels, groups, dtype, act="silu", eps=EPS)
    t = norm_inputs(channels, graphs, dtype, 5)
    fwd, bwd = both(norm, t, device)
    check_forward(norm, t, fwd, dtype, "silu")
    check_backward(norm, t, fwd[1], fwd[2], bwd, dtype, "silu")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["identity", "sigmoid", "tanh"])
def test_activations(device, act, dtype):
    norm = cg.group_norm_for(24, 3, dtype, act=act, eps=EPS)
    t = norm_inputs(24, [7, 60], dtype, 6)
    fwd, bwd = both(norm, t, device)
    check_forward(norm, t, fwd, dtype, act)
    check_backward(norm, t, fwd[1], fwd[2], bwd, dtype, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_mean_far_from_zero_costs_no_digits(device, dtype):
    """Values of 1000 +- 1: the bound holds a variance to the mean's own roundings, not to those of its square."""
    norm = cg.group_norm_for(16, 2, dtype, eps=EPS)
    t = norm_inputs(16, [3000, 5], dtype, 7)
    t["x"] = held(1000 + 8 * np.round(host(t["x"])), dtype)
    fwd, bwd = both(norm, t, device)
    check_forward(norm, t, fwd, dtype, "identity")
    _, r = ox.group_stats(host(t["x"]), t["ptr"], 2, EPS)
    assert np.abs(host(fwd[2]) / r - 1).max() < 1e-3


def test_without_weights_and_statistics(device):
    norm = cg.group_norm_for(12, 4, "f32", act="silu", eps=EPS)
    t = norm_inputs(12, [9, 0, 30], "f32", 8)
    t["w"], t["bias"] = real(np.ones(12), "f32"), real(np.zeros(12), "f32")
    d = {k: up(v, device) for k, v in t.items()}
    want = cg.group_norm_forward(norm, d["x"], d["ptr"], d["w"], d["bias"])
    y, mean, rstd = cg.group_norm_forward(norm, d["x"], d["ptr"], None, None, need_stats=False)
    assert mean is None and rstd is None and y.equal(want[0])
    a = cg.group_norm_backward(norm, d["x"], d["ptr"], None, None, want[1], want[2], d["dy"])
    b = cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], want[1], want[2], d["dy"])
    assert all(p.equal(q) for p, q in zip(a, b))
    for i in range(3):
        need = [j == i for j in range(3)]
        c = cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], want[1], want[2], d["dy"], need=need)
        assert [g is not None for g in c] == need and c[i].equal(b[i])


def test_rows_of_no_graph(device):
    """Left as they were in given tensors, zeros in new ones, whatever they hold; they do not reach the rest."""
    import torch
    norm = cg.group_norm_for(20, 4, "f32", act="tanh", eps=EPS)
    t = norm_inputs(20, [5, 300, 2], "f32", 9, outside=(70, 90))
    d = {k: up(v, device) for k, v in t.items()}
    want, grads = both(norm, t, device)
    assert not want[0][:70].any() and not want[0][-90:].any() and not grads[0][:70].any() and not grads[0][-90:].any()
    for v in (d["x"], d["dy"]):
        v[:70], v[-90:] = float("nan"), float("inf")
    y, gx = torch.full_like(d["x"], 7.0), torch.full_like(d["x"], 8.0)
    got = cg.group_norm_forward(norm, d["x"], d["ptr"], d["w"], d["bias"], y=y)
    back = cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], got[1], got[2], d["dy"], grad_x=gx)
    assert (y[:70] == 7).all() and (y[-90:] == 7).all() and (gx[:70] == 8).all() and (gx[-90:] == 8).all()
    assert y[70:-90].equal(want[0][70:-90]) and gx[70:-90].equal(grads[0][70:-90])
    assert got[1].equal(want[1]) and back[1].equal(grads[1]) and back[2].equal(grads[2])


def test_one_graph_not_finite(device):
    """A value that is not finite reaches its own graph and group alone (and the weights' gradients)."""
    norm = cg.group_norm_for(8, 2, "f32", eps=EPS)
    t = norm_inputs(8, [40, 40, 40], "f32", 10, outside=(0, 0))
    want, grads = both(norm, t, device)
    t["x"][50, 1] = float("inf")
    got, back = both(norm, t, device)
    assert not got[0][40:80, :4].isfinite().any() and got[0][40:80, 4:].equal(want[0][40:80, 4:])
    for part in (slice(0, 40), slice(80, 120)):
        assert got[0][part].equal(want[0][part]) and back[0][part].equal(grads[0][part])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_pitches_and_odd_addresses(device, dtype):
    """The first columns of wider rows, at any element."""
    import torch
    norm = cg.group_norm_for(37, 1, dtype, act="silu", eps=EPS)
    t = norm_inputs(37, [50, 3, 200], dtype, 11)
    d = {k: up(v, device) for k, v in t.items()}
    fwd, bwd = both(norm, t, device)
    n = d["x"].shape[0]

    def wide(v, ld, off):
        flat = torch.full((n * ld + off,), 3.0, dtype=d["x"].dtype, device=device)[off:].view(n, ld)
        rows = flat[:, :37]
        if v is not None:
            rows.copy_(v)
        return rows, flat
    x, dy = wide(d["x"], 41, 1)[0], wide(d["dy"], 64, 3)[0]
    (y, yf), (gx, gf) = wide(None, 39, 5), wide(None, 50, 0)
    cg.group_norm_forward(norm, x, d["ptr"], d["w"], d["bias"], y=y)
    got = cg.group_norm_backward(norm, x, d["ptr"], d["w"], d["bias"], fwd[1], fwd[2], dy, grad_x=gx)
    inside = slice(int(t["ptr"][0]), int(t["ptr"][-1]))
    assert y[inside].equal(fwd[0][inside]) and gx[inside].equal(bwd[0][inside]) and got[1].equal(bwd[1])
    assert (yf[:, 37:] == 3).all() and (gf[:, 37:] == 3).all()


def test_no_rows_and_no_graphs(device):
    import torch
    norm = cg.group_norm_for(6, 2, "f32", eps=EPS)
    x = torch.randn(5, 6, device=device)
    ptr = torch.zeros(1, dtype=torch.int32, device=device)
    y, mean, rstd = cg.group_norm_forward(norm, x[:0], torch.zeros(4, dtype=torch.int32, device=device), None, None)
    assert y.shape == (0, 6) and not mean.any() and torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5))
    y, mean, rstd = cg.group_norm_forward(norm, x, ptr, None, None)
    assert mean.shape == (0, 2)
    got = cg.group_norm_backward(norm, x, ptr, None, None, mean, rstd, x)
    assert not got[1].any() and not got[2].any()


def test_pointers_out_of_range_touch_nothing_else(device):
    """Row pointers past the rows, or falling, are read as if clamped to the rows: nothing outside is written."""
    import torch
    norm = cg.group_norm_for(16, 2, "f32", eps=EPS)
    buf = torch.full((3000, 16), 5.0, device=device)
    x, y = torch.randn(1000, 16, device=device), buf[1000:2000]
    for ptr in ([0, 500, 5000, 1 << 30], [-7, 300, 200, 1000], [900, 100, 100, -5], [2000, 3000, 4000, 5000]):
        p = torch.tensor(ptr, dtype=torch.int32, device=device)
        _, mean, rstd = cg.group_norm_forward(norm, x, p, None, None, y=y)
        cg.group_norm_backward(norm, x, p, None, None, mean, rstd, x, grad_x=y)
        torch.cuda.synchronize()
        assert (buf[:1000] == 5).all() and (buf[2000:] == 5).all(), ptr


def test_repeats_streams_and_graphs(device):
    """The same bits each time, on another stream, and from a captured graph whose inputs change."""
    import torch
    norm = cg.group_norm_for(48, 6, "f32", act="silu", eps=EPS)
    t = norm_inputs(48, [3, 2000, 0, 77], "f32", 12)
    d = {k: up(v, device) for k, v in t.items()}

    def run(stream=None):
        y, mean, rstd = cg.group_norm_forward(norm, d["x"], d["ptr"], d["w"], d["bias"], stream=stream)
        return (y, mean, rstd) + cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], mean, rstd, d["dy"],
                                                        stream=stream)
    want = run()
    assert all(a.equal(b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(a.equal(b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        d["x"].mul_(1.25).add_(0.5)
        d["dy"].neg_()
        d["ptr"][1:4] += 5
        graph.replay()
        got = [o.clone() for o in out]
        assert all(a.equal(b) for a, b in zip(got, run())), i


def test_more_graphs_than_workgroups(device):
    """Tens of thousands of graphs of a few rows, some empty: the backward's workgroups take several each."""
    norm = cg.group_norm_for(8, 2, "f32", act="silu", eps=EPS)
    sizes = list(np.random.default_rng(15).integers(0, 5, 20_000))
    t = norm_inputs(8, sizes, "f32", 15)
    fwd, bwd = both(norm, t, device)
    check_forward(norm, t, fwd, "f32", "silu")
    check_backward(norm, t, fwd[1], fwd[2], bwd, "f32", "silu")


def test_past_2_31_elements(device):
    """Rows past 2^31 elements: the last graph as if it stood alone."""
    import torch
    norm = cg.group_norm_for(64, 8, "bf16", act="silu", eps=EPS)
    n = (1 << 31) // 64 + 5000
    x = torch.empty((n, 64), dtype=torch.bfloat16, device=device)
    x[:-3000] = 1
    t = norm_inputs(64, [3000], "bf16", 13, outside=(0, 0))
    x[-3000:] = t["x"].to(device)
    ptr = torch.tensor([0, n - 3000, n], dtype=torch.int32, device=device)
    w, b = t["w"].to(device), t["bias"].to(device)
    y, mean, rstd = cg.group_norm_forward(norm, x, ptr, w, b)
    check_forward(norm, t, (y[-3000:], mean[1:], rstd[1:]), "bf16", "silu", rows=n)
    dy = torch.zeros_like(x)
    dy[-3000:] = t["dy"].to(device)
    gx, gw, gb = cg.group_norm_backward(norm, x, ptr, w, b, mean, rstd, dy)
    check_backward(norm, t, mean[1:], rstd[1:], (gx[-3000:], gw, gb), "bf16", "silu", rows=n)


def test_gradients_by_differences(device):
    import torch
    norm = cg.group_norm_for(6, 2, "f64", act="silu", eps=0.1)
    t = norm_inputs(6, [4, 0, 7], "f64", 14)
    d = {k: up(v, device) for k, v in t.items()}

    def loss(x, w, b):
        return (cg.group_norm_forward(norm, x, d["ptr"], w, b)[0] * d["dy"]).sum()
    args = [d["x"], d["w"], d["bias"]]
    _, mean, rstd = cg.group_norm_forward(norm, *[d[k] for k in ("x", "ptr", "w", "bias")])
    grads = cg.group_norm_backward(norm, d["x"], d["ptr"], d["w"], d["bias"], mean, rstd, d["dy"])
    h = 1e-5  # truncation h^2, cancellation 2^-53 / h: both below 1e-9 of sums of about 100
    gen = torch.Generator(device=device).manual_seed(0)
    for i, g in enumerate(grads):
        for _ in range(3):
            v = torch.randn(args[i].shape, dtype=torch.float64, device=device, generator=gen)
            lo, hi = list(args), list(args)
            lo[i], hi[i] = args[i] - h * v, args[i] + h * v
            assert abs((loss(*hi) - loss(*lo)).item() / (2 * h) - (g * v).sum().item()) < 1e-6
