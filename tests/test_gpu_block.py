"""Row norm and block join on the GPU against the float64 oracle, element by element, within bounds
that count roundings (block_cases); their edges, layouts, streams and graphs."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import block as ob
from oracle import wigner
from oracle.irreps import parse_irreps

from block_cases import (BROAD, CHANGING, CONFIGS, DTYPES, EPS, LADDER, ODD, ROW, SHAPES, WIDE, bound, inputs,
                         weight_roundings, wide)

pytestmark = pytest.mark.gpu

GRADS = ("grad_res", "grad_f", "grad_gate", "grad_w_post", "grad_scale", "grad_w_next")
ALPHA = 0.75


def up(t, device):
    return {k: None if v is None else v.to(device) for k, v in t.items()}


def make(irreps, dtype, config):
    gate, act, post, nxt = config
    return cg.block_for(irreps, dtype, gate=gate, act=act, post_norm=post, next_norm=nxt, eps=EPS, alpha=ALPHA)


def check(name, got, want, dtype, roundings, stored=True):
    value, size = want
    got = got.detach().double().cpu().numpy().reshape(value.shape)
    off = np.abs(got - value)
    most = bound(value, size, dtype, roundings, stored)
    assert np.all(off <= most), f"{name}: {np.max(off / np.maximum(most, 1e-300)):.3g} of the bound"


def run_join(block, d, **kw):
    h, u, rf, rh = cg.join_forward(block, d["res"], d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"])
    grads = cg.join_backward(block, d["dh"], d["du"] if block.next_norm else None, h, d["f"], d["gate"], d["w_post"],
                             d["scale"], d["w_next"], rf, rh, **kw)
    return (h, u, rf, rh), grads


def check_join(irreps, rows, dtype, config, device, seed):
    gate, act, post, nxt = config
    t = inputs(irreps, rows, dtype, config, seed)
    d, n = up(t, device), {k: wide(v) for k, v in t.items()}
    block = make(irreps, dtype, config)
    (h, u, rf, rh), grads = run_join(block, d)
    want = ob.join(irreps, n["res"], n["f"], n["gate"], n["w_post"], n["scale"], n["w_next"], EPS, ALPHA, act, post, nxt)
    check("h", h, want["h"], dtype, ROW)
    if nxt:
        check("u", u, want["u"], dtype, ROW)
        check("rstd_h", rh, want["rstd_h"], dtype, ROW, stored=False)
    else:
        assert u is None and rh is None
    if post:
        check("rstd_f", rf, want["rstd_f"], dtype, ROW, stored=False)
    host = lambda x: None if x is None else x.double().cpu().numpy()  # noqa: E731
    want = ob.join_grad(irreps, n["dh"], n["du"], host(h), n["f"], n["gate"], n["w_post"], n["scale"], n["w_next"],
                        host(rf), host(rh), ALPHA, act, post, nxt)
    for name, g in zip(GRADS, grads):
        assert (g is not None) == (name in want), name
        if g is not None:
            whole = name in ("grad_w_post", "grad_scale", "grad_w_next")
            check(name, g, want[name], dtype, weight_roundings(rows) if whole else ROW, stored=not whole)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("irreps, rows", SHAPES)
def test_norm(device, irreps, rows, dtype):
    t = inputs(irreps, rows, dtype, CONFIGS[0], 11)
    d, n = up(t, device), {k: wide(v) for k, v in t.items()}
    block = cg.block_for(irreps, dtype, eps=EPS)
    u, rstd = cg.norm_forward(block, d["x"], d["w"])
    want = ob.norm(irreps, n["x"], n["w"], EPS)
    check("u", u, want["u"], dtype, ROW)
    check("rstd", rstd, want["rstd"], dtype, ROW, stored=False)
    r = rstd.double().cpu().numpy()
    for add in (None, "add"):
        dx, dw = cg.norm_backward(block, d["x"], d["w"], rstd, d["du"], grad_add=add and d[add])
        want = ob.norm_grad(irreps, n["x"], n["w"], r, n["du"], add and n[add])
        check("grad_x", dx, want["grad_x"], dtype, ROW)
        check("grad_w", dw, want["grad_w"], dtype, weight_roundings(rows), stored=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("config", CONFIGS, ids=lambda c: "-".join(map(str, c)))
def test_join_configurations(device, config, dtype):
    check_join(ODD, 70, dtype, config, device, 21)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("irreps, rows", SHAPES)
def test_join_shapes(device, irreps, rows, dtype):
    check_join(irreps, rows, dtype, CONFIGS[0], device, 22)


@pytest.mark.parametrize("irreps, rows, dtype", WIDE)
def test_join_wide_scalar_rows(device, irreps, rows, dtype):
    for config in (CONFIGS[0], CONFIGS[3], CONFIGS[5]):
        check_join(irreps, rows, dtype, config, device, 23)


@pytest.mark.parametrize("dtype", DTYPES)
def test_join_with_a_degree_for_every_channel(device, dtype):
    for config in (CONFIGS[0], CONFIGS[3]):
        check_join(CHANGING, 300, dtype, config, device, 24)


def test_join_whose_sums_fill_the_lds(device):
    for config in (CONFIGS[3], CONFIGS[5]):
        check_join(BROAD, 4, "f32", config, device, 25)


def test_rows_with_a_pitch_side_by_side_and_unaligned(device):
    """f and its gates in one buffer that starts at an odd element, their gradients in another: the
    same bits as from separate tensors, and nothing written beside the rows."""
    import torch
    for irreps, dtype in ((ODD, "bf16"), ("32x0e+32x1o+32x2e", "f32"), ("257x0e", "f16")):
        t = inputs(irreps, 33, dtype, CONFIGS[0], 31)
        d = up(t, device)
        block = make(irreps, dtype, CONFIGS[0])
        w, c = block.d, block.channels
        (h, u, rf, rh), grads = run_join(block, d)
        wide_buf = lambda: torch.full((33 * (w + c + 5) + 3,), 7.0, dtype=block.torch_dtype,  # noqa: E731
                                      device=device)[3:].view(33, w + c + 5)
        buf, out = wide_buf(), wide_buf()
        buf[:, :w], buf[:, w + 1:w + 1 + c] = d["f"], d["gate"]
        d2 = {**d, "f": buf[:, :w], "gate": buf[:, w + 1:w + 1 + c]}
        (h2, u2, rf2, rh2), grads2 = run_join(block, d2, outs=(None, out[:, :w], out[:, w + 1:w + 1 + c], None, None,
                                                               None))
        for a, b in zip((h, u, rf, rh, *grads), (h2, u2, rf2, rh2, *grads2)):
            assert torch.equal(a, b)
        assert torch.all(out[:, w] == 7) and torch.all(out[:, w + 1 + c:] == 7)
        # the norm's rows with a pitch
        nb = cg.block_for(irreps, dtype, eps=EPS)
        buf[:, :w] = d["x"]
        a, b = cg.norm_forward(nb, d["x"], d["w"]), cg.norm_forward(nb, buf[:, :w], d["w"])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_outputs_end_where_their_rows_end(device):
    """Outputs inside larger buffers: what lies before and behind them is left alone."""
    import torch
    for irreps, rows, dtype in ((ODD, 1, "f16"), ("3x0e+2x2e+5x0o", 6, "bf16"), ("257x0e", 3, "f32"), (LADDER, 2, "f64")):
        t = inputs(irreps, rows, dtype, CONFIGS[0], 41)
        d = up(t, device)
        block = make(irreps, dtype, CONFIGS[0])
        held = []

        def inside(shape, ty):
            n = int(np.prod(shape))
            big = torch.full((n + 512,), 3.0, dtype=ty, device=device)
            held.append((big, n))
            return big[256:256 + n].view(shape)
        dt, rt, c = block.torch_dtype, block.real_dtype, block.channels
        h, u, rf, rh = cg.join_forward(block, d["res"], d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"],
                                       h=inside((rows, block.d), dt), u=inside((rows, block.d), dt),
                                       rstd_f=inside((rows,), rt), rstd_h=inside((rows,), rt))
        need = cg.block_workspace_size(block, rows)
        ws = torch.full((need + 512,), 9, dtype=torch.uint8, device=device)
        cg.join_backward(block, d["dh"], d["du"], h, d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"], rf, rh,
                         outs=(inside((rows, block.d), dt), inside((rows, block.d), dt), inside((rows, c), dt),
                               inside((c,), rt), inside((c,), rt), inside((c,), rt)), workspace=ws[256:256 + need])
        torch.cuda.synchronize()
        for big, n in held:
            assert torch.all(big[:256] == 3) and torch.all(big[256 + n:] == 3)
        assert torch.all(ws[:256] == 9) and torch.all(ws[256 + need:] == 9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_weights_left_out_are_ones(device, dtype):
    import torch
    t = inputs(ODD, 20, dtype, CONFIGS[0], 51)
    d = up(t, device)
    block = make(ODD, dtype, CONFIGS[0])
    ones = torch.ones(block.channels, dtype=block.real_dtype, device=device)
    a = run_join(block, {**d, "w_post": None, "scale": None, "w_next": None})
    b = run_join(block, {**d, "w_post": ones, "scale": ones, "w_next": ones})
    for x, y in zip((*a[0], *a[1]), (*b[0], *b[1])):
        assert torch.equal(x, y)
    # a missing gradient of h is a zero one
    h, u, rf, rh = a[0]
    args = (d["du"], h, d["f"], d["gate"], None, None, None, rf, rh)
    for x, y in zip(cg.join_backward(block, None, *args), cg.join_backward(block, torch.zeros_like(h), *args)):
        assert torch.equal(x, y)


def test_subsets_of_gradients_have_the_same_bits(device):
    import torch
    t = inputs(ODD, 40, "f32", CONFIGS[0], 52)
    d = up(t, device)
    block = make(ODD, "f32", CONFIGS[0])
    (h, u, rf, rh), full = run_join(block, d)
    args = (d["dh"], d["du"], h, d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"], rf, rh)
    for k in range(6):
        need = tuple(i == k for i in range(6))
        got = cg.join_backward(block, *args, need=need)
        assert torch.equal(got[k], full[k]) and all(g is None for i, g in enumerate(got) if i != k)
    nb = cg.block_for(ODD, "f32", eps=EPS)
    rstd = cg.norm_forward(nb, d["x"], d["w"])[1]
    dx, dw = cg.norm_backward(nb, d["x"], d["w"], rstd, d["du"])
    assert torch.equal(cg.norm_backward(nb, d["x"], d["w"], rstd, d["du"], need=(True, False))[0], dx)
    assert torch.equal(cg.norm_backward(nb, d["x"], d["w"], rstd, d["du"], need=(False, True))[1], dw)


def test_a_row_that_is_not_finite_stays_alone(device):
    """NaN and infinities in some rows, the last among them (the lanes past the end work on it): the
    other rows have the bits that they have without."""
    import torch
    for irreps, rows in ((ODD, 37), ("32x0e+32x1o+32x2e", 21), (LADDER, 5)):
        t = inputs(irreps, rows, "f32", CONFIGS[0], 61)
        d = up(t, device)
        block = make(irreps, "f32", CONFIGS[0])
        clean, cgrads = run_join(block, d)
        bad = [1, rows - 1]
        for key, value in (("f", float("nan")), ("res", float("inf")), ("gate", float("nan")), ("du", -float("inf"))):
            d2 = {**d, key: d[key].clone()}
            d2[key][bad, -1] = value
            got, grads = run_join(block, d2)
            keep = [r for r in range(rows) if r not in bad]
            for a, b in zip((*got, *grads[:3]), (*clean, *cgrads[:3])):
                assert torch.equal(a[keep], b[keep]), key
            assert not torch.isfinite(grads[5] if key == "du" else grads[4]).all()


def test_zero_rows_and_no_rows(device):
    import torch
    block = make(ODD, "f32", CONFIGS[0])
    nb = cg.block_for(ODD, "f32", eps=EPS)
    z = torch.zeros(5, block.d, device=device)
    w = torch.ones(block.channels, device=device)
    u, rstd = cg.norm_forward(nb, z, w)
    assert not u.any() and torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5))
    dx, dw = cg.norm_backward(nb, z, w, rstd, torch.ones_like(z))
    assert torch.allclose(dx, torch.full_like(dx, EPS ** -0.5)) and not dw.any()
    e = torch.empty(0, block.d, device=device)
    eg, er = torch.empty(0, block.channels, device=device), torch.empty(0, device=device)
    h, u, rf, rh = cg.join_forward(block, e, e, eg, w, w, w)
    assert h.shape == e.shape and u.shape == e.shape
    grads = cg.join_backward(block, e, e, h, e, eg, w, w, w, rf, rh,
                             outs=(None, None, None) + tuple(torch.full_like(w, 5) for _ in range(3)))
    assert all(not g.any() for g in grads[3:])
    assert not cg.norm_backward(nb, e, w, er, e, grad_w=torch.full_like(w, 5))[1].any()


def test_gradients_against_differences(device):
    """float64: the change of the forward's own outputs along a direction."""
    import torch
    for config in (CONFIGS[0], CONFIGS[2], CONFIGS[3]):
        t = inputs(ODD, 9, "f64", config, 71)
        t["f"][4] += 0.5  # away from the zero row, where the norm's curvature is 1 / eps
        d = up(t, device)
        block = make(ODD, "f64", config)
        (h, u, rf, rh), grads = run_join(block, d)
        names = ("res", "f", "gate", "w_post", "scale", "w_next")
        gen = torch.Generator().manual_seed(1)
        step = 1e-6
        for name, g in zip(names, grads):
            if g is None:
                continue
            way = torch.randn(d[name].shape, generator=gen, dtype=torch.float64).to(device)

            def loss(sign):
                x = {**d, name: d[name] + sign * step * way}
                a, b, _, _ = cg.join_forward(block, x["res"], x["f"], x["gate"], x["w_post"], x["scale"], x["w_next"])
                return ((a * d["dh"]).sum() + ((b * d["du"]).sum() if block.next_norm else 0)).item()
            num, ana = (loss(1) - loss(-1)) / (2 * step), (g * way).sum().item()
            # rounding of the losses (about 1e3, over the step) and the third derivative's term
            assert abs(num - ana) <= 1e-5 * (1 + abs(ana)), name


def test_norm_and_join_commute_with_rotations(device):
    import torch
    rng = np.random.default_rng(3)
    irr = "5x0e+4x1o+3x2e+1x3o"
    big = torch.from_numpy(wigner.irreps_d(parse_irreps(irr), wigner.random_rotation(rng))).to(device)
    d = up(inputs(irr, 12, "f64", CONFIGS[0], 81), device)
    block = make(irr, "f64", CONFIGS[0])
    turn = lambda a: (a @ big.t().contiguous()).contiguous()  # noqa: E731
    a, ga = run_join(block, d)
    b, gb = run_join(block, {**d, **{k: turn(d[k]) for k in ("res", "f", "dh", "du")}})
    for x, y in ((turn(a[0]), b[0]), (turn(a[1]), b[1]), (turn(ga[0]), gb[0]), (turn(ga[1]), gb[1]),
                 *zip(ga[2:], gb[2:])):
        assert torch.allclose(x, y, rtol=1e-9, atol=1e-9)


def test_rows_past_two_to_the_31(device):
    """Offsets of 64 bits: the last rows of a tensor of 2.2e9 elements have the bits that they have alone."""
    import torch
    irreps, rows = "2048x0e", 1_070_000
    block = cg.block_for(irreps, "bf16", eps=EPS)
    x = torch.empty(rows, block.d, dtype=torch.bfloat16, device=device)
    x.fill_(0.5)
    gen = torch.Generator(device=device).manual_seed(2)
    x[-40:] = torch.randn(40, block.d, generator=gen, device=device).to(torch.bfloat16)
    u, rstd = cg.norm_forward(block, x, None)
    u2, rstd2 = cg.norm_forward(block, x[-40:].clone(), None)
    assert torch.equal(u[-40:], u2) and torch.equal(rstd[-40:], rstd2)
    dx, dw = cg.norm_backward(block, x, None, rstd, u, grad_x=x.new_empty(x.shape))
    dx2, _ = cg.norm_backward(block, x[-40:].clone(), None, rstd2, u2)
    assert torch.equal(dx[-40:], dx2) and torch.isfinite(dw).all()
    del dx
    join = make(irreps, "bf16", CONFIGS[0])
    small = x[-40:].clone()
    h, v, rf, rh = cg.join_forward(join, x, u, u, None, None, None)
    h2, v2, rf2, rh2 = cg.join_forward(join, small, u2, u2, None, None, None)
    assert torch.equal(h[-40:], h2) and torch.equal(v[-40:], v2) and torch.equal(rh[-40:], rh2)
    need = (True, True, True, False, False, False)
    got = cg.join_backward(join, x, u, h, u, u, None, None, None, rf, rh, need=need)
    want = cg.join_backward(join, small, u2, h2, u2, u2, None, None, None, rf2, rh2, need=need)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[-40:], b)


def test_same_bits_again_on_another_stream_and_in_a_graph(device):
    """Two eager calls, a call on a side stream with inputs made there, and replays of a captured step
    with new inputs and eager work between them: all bitwise equal."""
    import torch
    irreps = "32x0e+32x1o+32x2e"
    d = up(inputs(irreps, 700, "f32", CONFIGS[0], 91), device)
    block = make(irreps, "f32", CONFIGS[0])
    nb = cg.block_for(irreps, "f32", eps=EPS)

    def step(t, **kw):
        u0, r0 = cg.norm_forward(nb, t["x"], t["w"], **kw)
        h, u, rf, rh = cg.join_forward(block, t["x"], t["f"], t["gate"], t["w_post"], t["scale"], t["w_next"], **kw)
        grads = cg.join_backward(block, t["dh"], t["du"], h, t["f"], t["gate"], t["w_post"], t["scale"], t["w_next"],
                                 rf, rh, **kw)
        dx, dw = cg.norm_backward(nb, t["x"], t["w"], r0, t["du"], grad_add=grads[0], **kw)
        return (u0, r0, h, u, rf, rh, *grads, dx, dw)
    first = [t.clone() for t in step(d)]
    torch.cuda.synchronize()
    for a, b in zip(first, step(d)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine = {k: v.clone() for k, v in d.items()}
        got = step(mine)
    side.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)
    # a stream given by hand, the tensors on the current one
    side.wait_stream(torch.cuda.current_stream())
    got = cg.norm_forward(nb, d["x"], d["w"], stream=side)
    side.synchronize()
    assert torch.equal(got[0], first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(d)
    torch.cuda.synchronize()
    for rep in range(3):
        if rep:
            d["x"].copy_(torch.randn(d["x"].shape, device=device))
            d["gate"].copy_(torch.randn(d["gate"].shape, device=device))
        want = [t.clone() for t in step(d)]
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), f"replay {rep}"


def test_closed_handles_are_refused(device):
    import torch
    b, o = cg.Block("4x0e", "f32"), cg.AdamW([4])
    x, p = torch.zeros(3, 4, device=device), torch.zeros(4, device=device)
    m, v, _, _ = o.state(device)
    cg.norm_forward(b, x, None)
    torch.cuda.synchronize()   # a block's kernels end before their code is unloaded
    b.close()
    o.close()
    with pytest.raises(cg.CgtpError, match="block is NULL"):
        cg.norm_forward(b, x, None)
    with pytest.raises(cg.CgtpError, match="NULL"):
        cg.adamw_step(o, [p], [p.clone()], m, v, step=1)
