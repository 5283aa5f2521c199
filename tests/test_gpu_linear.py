"""Experts' products on the GPU against the float64 oracle, element by element, within bounds that count roundings
(expert_cases); masks, layouts, streams, graphs, and the run of norm, routing and products."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import experts as ox

from block_cases import work_unit
from expert_cases import DTYPES, LINEAR_CASES, held, host, linear_bounds, linear_inputs, real, within

pytestmark = pytest.mark.gpu


def up(a, device):
    import torch
    return None if a is None else (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(device)


def make(a, b, e, k, dtype, t, device):
    """The linear, its device tensors and the order."""
    linear = cg.linear_for(a, b, dtype, experts=e, top_k=k)
    d = {n: up(v, device) for n, v in t.items()}
    order = cg.route_order(cg.router_for(e, k, "f32"), d["experts"]) if k else None
    return linear, d, order


def run(linear, d, order, **kw):
    out = cg.linear_forward(linear, d["x"], d["w"], d["experts"], d["weights"], order)
    return (out,) + cg.linear_backward(linear, d["x"], d["w"], d["g"], d["experts"], d["weights"], order, **kw)


def check(a, b, e, k, n, dtype, t, got):
    want = ox.linear(a, b, host(t["x"]), host(t["w"]), t["experts"], None if t["weights"] is None else host(t["weights"]),
                     host(t["g"]))
    slots = n if not k else max(int((t["experts"] == i).sum()) for i in range(e))
    f, x, p, w = linear_bounds(a, b, dtype, k, slots)
    # fp16 products p g below its normal range are off by half its spacing there, times |x|
    tiny = 2.0 ** -25 * slots * 15 * np.abs(host(t["x"])).max() if dtype == "f16" and k else 0
    for name, g, roundings, stored, extra in (("out", got[0], f, dtype, 0), ("grad_x", got[1], x, dtype, 0),
                                              ("grad_w", got[2], w, dtype, tiny), ("grad_weights", got[3], p, None, 0)):
        if k or name != "grad_weights":
            value, size = want[name]
            within(name, g, value, roundings * size + extra + (work_unit(dtype) * np.abs(value) if stored is None else 0), stored)
    assert k or got[3] is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("a, b, e, k, n", LINEAR_CASES)
def test_shapes(device, a, b, e, k, n, dtype):
    t = linear_inputs(a, b, e, k, n, dtype, 41)
    linear, d, order = make(a, b, e, k, dtype, t, device)
    got = run(linear, d, order)
    check(a, b, e, k, n, dtype, t, got)
    # the rows' order changes no bit; nor does leaving outputs out
    if k:
        plain = (None,) + tuple(order[1:])
        assert all(p.equal(q) for p, q in zip(run(linear, d, plain), got))
    for i in range(3):
        need = [j == i for j in range(3)]
        part = cg.linear_backward(linear, d["x"], d["w"], d["g"], d["experts"], d["weights"], order, need=need)
        assert [p is not None for p in part] == [m and (j < 2 or k > 0) for j, m in enumerate(need)]
        assert part[i] is None or part[i].equal(got[1 + i])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(device, dtype):
    """Stretches of several lengths, and experts with a large, a small and no share."""
    a = "16x0e+16x1o"
    t = linear_inputs(a, a, 4, 2, 30_000, dtype, 42)
    t["experts"][:, 0] = 1
    t["experts"][:, 1] = np.where(np.arange(30_000) % 4099 == 7, 3, -1)
    linear, d, order = make(a, a, 4, 2, dtype, t, device)
    got = run(linear, d, order)
    check(a, a, 4, 2, 30_000, dtype, t, got)
    assert not got[2][0].any() and not got[2][2].any()


def test_what_a_row_has_not_chosen_does_not_reach_it(device):
    """Weights of an expert that are not finite, and rows that are not, beside rows that take neither."""
    a = "20x0e+9x1o"
    t = linear_inputs(a, a, 4, 2, 200, "f32", 43, free=False)
    rng = np.random.default_rng(1)
    t["experts"] = np.argsort(rng.random((200, 3)), axis=1)[:, :2].astype(np.int32)  # 3 is free
    t["experts"][17], t["experts"][90] = (3, 0), (1, -1)
    linear, d, order = make(a, a, 4, 2, "f32", t, device)
    want = run(linear, d, order)
    d["w"][3], d["x"][17], d["g"][17] = float("nan"), float("inf"), float("nan")
    got = run(linear, d, order)
    rest = [i for i in range(200) if i != 17]
    for i in (0, 1, 3):
        assert got[i][rest].equal(want[i][rest]) and not got[i][17].isfinite().all()
    assert got[2][1:3].equal(want[2][1:3])   # experts that row 17 has not chosen


def test_rows_without_an_expert(device):
    import torch
    a, b = "7x0e+5x1o", "5x1o+9x0e"
    t = linear_inputs(a, b, 3, 2, 50, "bf16", 44)
    t["experts"][:] = -1
    t["experts"][3] = (5, -2)
    linear, d, order = make(a, b, 3, 2, "bf16", t, device)
    d["x"][:] = float("nan")
    for got in run(linear, d, order):
        assert not got.any()
    t["experts"][10] = (1, 1)  # named twice: counted twice
    t["x"][:] = 1
    linear, d, order = make(a, b, 3, 2, "bf16", t, device)
    got = run(linear, d, order)
    check(a, b, 3, 2, 50, "bf16", t, got)
    assert got[3][10, 0] == got[3][10, 1] != 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_pitches_and_odd_addresses(device, dtype):
    import torch
    a, b = "19x0e+7x1o", "7x1o+10x0e"
    t = linear_inputs(a, b, 3, 2, 60, dtype, 45)
    linear, d, order = make(a, b, 3, 2, dtype, t, device)
    want = run(linear, d, order)

    def wide(v, cols, ld, off):
        flat = torch.full((60 * ld + off,), 3.0, dtype=d["x"].dtype, device=device)[off:].view(60, ld)
        if v is not None:
            flat[:, :cols].copy_(v)
        return flat[:, :cols], flat
    x, g = wide(d["x"], 40, 43, 1)[0], wide(d["g"], 31, 64, 3)[0]
    w = torch.empty(d["w"].numel() + 1, dtype=d["w"].dtype, device=device)[1:].view_as(d["w"]).copy_(d["w"])
    (out, of), (gx, gf) = wide(None, 31, 33, 5), wide(None, 40, 41, 0)
    cg.linear_forward(linear, x, w, d["experts"], d["weights"], order, out=out)
    got = cg.linear_backward(linear, x, w, g, d["experts"], d["weights"], order, outs=(gx, None, None))
    assert out.equal(want[0]) and gx.equal(want[1]) and got[1].equal(want[2]) and got[2].equal(want[3])
    assert (of[:, 31:] == 3).all() and (gf[:, 40:] == 3).all()


def test_lists_out_of_range_touch_nothing_else(device):
    """Entries of the lists that are no rows or slots are passed over."""
    import torch
    a = "8x0e+8x1o"
    t = linear_inputs(a, a, 4, 2, 100, "f32", 46)
    linear, d, order = make(a, a, 4, 2, "f32", t, device)
    rows, slots, offsets = (o.clone() for o in order)
    rows[::3] = torch.tensor([-1, 100, 1 << 30, -(1 << 31)], device=device, dtype=torch.int32).repeat(9)[:34]
    slots[::2], slots[1::4] = 1 << 30, -7
    for off in (offsets, torch.tensor([-5, 90, 20, 1 << 30, -9], dtype=torch.int32, device=device)):
        buf = torch.full((300, linear.d_in), 5.0, device=device)
        bad = (rows, slots, off)
        cg.linear_forward(linear, d["x"], d["w"], d["experts"], d["weights"], bad, out=buf[100:200])
        cg.linear_backward(linear, d["x"], d["w"], d["g"], d["experts"], d["weights"], bad, outs=(buf[100:200], None, None))
        torch.cuda.synchronize()
        assert (buf[:100] == 5).all() and (buf[200:] == 5).all()


def test_no_rows(device):
    import torch
    linear = cg.linear_for("4x0e", "6x0e", "f32", experts=3, top_k=1)
    x, w, i32 = torch.empty(0, 4, device=device), torch.randn(3, 24, device=device), torch.int32
    e, p = torch.empty(0, 1, dtype=i32, device=device), torch.empty(0, 1, device=device)
    order = cg.route_order(cg.router_for(3, 1), e)
    assert cg.linear_forward(linear, x, w, e, p, order).shape == (0, 6)
    gx, gw, gp = cg.linear_backward(linear, x, w, torch.empty(0, 6, device=device), e, p, order)
    assert gx.shape == (0, 4) and gp.shape == (0, 1) and not gw.any()


def test_past_2_31_elements(device):
    """Rows and slots past 2^31 elements: the last ones as if they stood alone."""
    import torch
    a, e, k, dtype = "64x0e", 3, 1, "bf16"
    n, tail = (1 << 31) // 64 + 5000, 3000
    t = linear_inputs(a, a, e, k, tail, dtype, 47, free=False)
    linear = cg.linear_for(a, a, dtype, experts=e, top_k=k)
    d = {m: up(v, device) for m, v in t.items()}
    big = {m: torch.zeros((n, d[m].shape[1]), dtype=d[m].dtype, device=device) for m in ("x", "g", "weights")}
    big["experts"] = torch.full((n, k), -1, dtype=torch.int32, device=device)
    for m in big:
        big[m][-tail:] = d[m]
    big["w"] = d["w"]
    order = cg.route_order(cg.router_for(e, k), big["experts"])
    got = run(linear, big, order)
    assert not got[0][:1000].any()
    check(a, a, e, k, tail, dtype, t, (got[0][-tail:], got[1][-tail:], got[2], got[3][-tail:]))


def layer(device, dtype, n=3000, seed=48):
    """Tensors of a layer: features of graphs, their norm, the router's head, the experts."""
    import torch
    gen = torch.Generator(device=device).manual_seed(seed)
    td = {"f32": torch.float32, "f64": torch.float64}[dtype]
    normal = lambda *s: torch.randn(*s, generator=gen, device=device, dtype=td)  # noqa: E731
    irreps = "24x0e+8x1o+4x2e"
    p = {"norm": cg.group_norm_for(24, 3, dtype, act="silu", eps=1e-5), "head": cg.linear_for("24x0e", "8x0e", dtype),
         "router": cg.router_for(8, 2, dtype), "linear": cg.linear_for(irreps, irreps, dtype, experts=8, top_k=2)}
    t = {"x": normal(n, 68), "w": 1 + 0.1 * normal(24), "b": 0.1 * normal(24), "head": 0.3 * normal(1, 24 * 8),
         "experts": 0.2 * normal(8, p["linear"].weight_numel), "g": normal(n, 68),
         "ptr": torch.tensor([0, n // 7, n // 7, n // 2, n], dtype=torch.int32, device=device)}
    return p, t


def layer_forward(p, t):
    s = t["x"][:, :24]
    h, mean, rstd = cg.group_norm_forward(p["norm"], s, t["ptr"], t["w"], t["b"])
    logits = cg.linear_forward(p["head"], h, t["head"])
    e, q = cg.route_forward(p["router"], logits)
    order = cg.route_order(p["router"], e)
    return cg.linear_forward(p["linear"], t["x"], t["experts"], e, q, order), (h, mean, rstd, logits, e, q, order)


def layer_backward(p, t, kept):
    h, mean, rstd, logits, e, q, order = kept
    gx, ge, gq = cg.linear_backward(p["linear"], t["x"], t["experts"], t["g"], e, q, order)
    gl = cg.route_backward(p["router"], logits, e, gq)
    gh, ghead, _ = cg.linear_backward(p["head"], h, t["head"], gl)
    gs, gw, gb = cg.group_norm_backward(p["norm"], t["x"][:, :24], t["ptr"], t["w"], t["b"], mean, rstd, gh)
    gx[:, :24] += gs
    return {"x": gx, "w": gw, "b": gb, "head": ghead, "experts": ge}


def test_a_layer_and_its_gradients_by_differences(device):
    """Norm, head, routing and products as they are used together, in double."""
    import torch
    p, t = layer(device, "f64", n=60)
    out, kept = layer_forward(p, t)
    grads = layer_backward(p, t, kept)
    gen = torch.Generator(device=device).manual_seed(1)
    h = 1e-6  # truncation h^2; cancellation 2^-53 / h of sums of about 1e3: both below 1e-6
    for name, g in grads.items():
        v = torch.randn(g.shape, generator=gen, device=device, dtype=torch.float64)
        sides = []
        for s in (h, -h):
            o, k = layer_forward(p, {**t, name: t[name] + s * v})
            assert k[4].equal(kept[4])      # the choice stays: the differences are of one smooth piece
            sides.append((o * t["g"]).sum().item())
        assert abs((sides[0] - sides[1]) / (2 * h) - (g * v).sum().item()) < 1e-4, name


def test_a_layer_captured_and_on_another_stream(device):
    """A captured forward and backward, replayed on changing inputs beside eager work, and on another stream."""
    import torch
    p, t = layer(device, "f32")

    def step():
        out, kept = layer_forward(p, t)
        return [out] + list(layer_backward(p, t, kept).values())
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(a.equal(b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        t["x"].copy_(torch.randn_like(t["x"]))
        t["g"].copy_(torch.randn_like(t["g"]))
        t["ptr"][2] += 3
        graph.replay()
        got = [o.clone() for o in outs]
        assert all(a.equal(b) for a, b in zip(got, step())), i


def test_two_captured_layers_replayed_at_once(device):
    """Two graphs of one configuration, each with its own workspaces, on two streams."""
    import torch
    graphs, outs, wants, streams = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    layers = [layer(device, "f32", n, seed) for n, seed in ((20000, 1), (9001, 2))]

    def step(p, t):
        out, kept = layer_forward(p, t)
        return [out] + list(layer_backward(p, t, kept).values())
    for p, t in layers:
        wants.append([v.clone() for v in step(p, t)])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(p, t))
    for _ in range(3):
        for o in outs:
            for v in o:
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert all(a.equal(b) for a, b in zip(o, w))
