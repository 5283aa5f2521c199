"""The oracle's norm, join and AdamW against torch autograd and torch.optim on the CPU in float64,
against central differences, and their invariances."""
import numpy as np
import pytest

from oracle import block as ob
from oracle import optim as oo
from oracle import wigner
from oracle.irreps import parse_irreps

from block_cases import CONFIGS, EPS, ODD, inputs, wide


def plain_join(t, deg, gate, kind, alpha):
    import torch
    spread = lambda c: torch.repeat_interleave(c, torch.from_numpy(deg), dim=-1)  # noqa: E731
    normed = lambda x: x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + EPS)       # noqa: E731
    y = t["f"] if t["w_post"] is None else normed(t["f"]) * spread(t["w_post"])
    y = y * spread(t["scale"])
    if gate is not None:
        a = {"identity": lambda g: g, "tanh": torch.tanh, "sigmoid": torch.sigmoid,
             "silu": torch.nn.functional.silu}[kind](t["gate"])
        y = y * (a if a.shape[1] == 1 else spread(a))
    h = alpha * t["res"] + y
    return h, None if t["w_next"] is None else normed(h) * spread(t["w_next"])


@pytest.mark.parametrize("config", CONFIGS)
def test_join_and_its_gradient_against_autograd(config):
    gate, kind, post, nxt = config
    t = inputs(ODD, 6, "f64", config, 3)
    deg = ob.degrees(ODD)
    leaves = {k: t[k].clone().requires_grad_() for k in ("res", "f", "gate", "w_post", "scale", "w_next")
              if t[k] is not None}
    live = {**t, **leaves}
    h, u = plain_join(live, deg, gate, kind, 0.75)
    n = {k: wide(v) for k, v in t.items()}
    fwd = ob.join(ODD, n["res"], n["f"], n["gate"], n["w_post"], n["scale"], n["w_next"], EPS, 0.75, kind, post, nxt)
    np.testing.assert_allclose(fwd["h"][0], h.detach().numpy(), rtol=1e-13, atol=1e-13)
    loss = (h * t["dh"]).sum()
    if nxt:
        np.testing.assert_allclose(fwd["u"][0], u.detach().numpy(), rtol=1e-13, atol=1e-13)
        loss = loss + (u * t["du"]).sum()
    loss.backward()
    got = ob.join_grad(ODD, n["dh"], n["du"], fwd["h"][0], n["f"], n["gate"], n["w_post"], n["scale"], n["w_next"],
                       ob.rstd(n["f"], EPS), ob.rstd(fwd["h"][0], EPS), 0.75, kind, post, nxt)
    for k, leaf in leaves.items():
        want, size = leaf.grad.numpy(), got["grad_" + k][1]
        assert np.all(np.abs(got["grad_" + k][0] - want) <= 1e-13 * size + 1e-300), k


def test_norm_gradient_against_differences_and_autograd():
    rng = np.random.default_rng(0)
    x, w, du = rng.standard_normal((3, 65)), 1 + 0.1 * rng.standard_normal(31), rng.standard_normal((3, 65))
    got = ob.norm_grad(ODD, x, w, ob.rstd(x, EPS), du)
    loss = lambda a, b: (ob.norm(ODD, a, b, EPS)["u"][0] * du).sum()  # noqa: E731
    step = 1e-6
    for k in range(20):
        i, j, c = rng.integers(3), rng.integers(65), rng.integers(31)
        e, ew = np.zeros_like(x), np.zeros_like(w)
        e[i, j], ew[c] = step, step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - got["grad_x"][0][i, j]) < 1e-8
        assert abs((loss(x, w + ew) - loss(x, w - ew)) / (2 * step) - got["grad_w"][0][c]) < 1e-8


def test_norm_and_join_commute_with_rotations():
    rng = np.random.default_rng(4)
    irr = "3x0e+2x1o+2x2e"
    big = wigner.irreps_d(parse_irreps(irr), wigner.random_rotation(rng))
    t = {k: wide(v) for k, v in inputs(irr, 4, "f64", CONFIGS[0], 5).items()}
    turn = lambda a: a @ big.T  # noqa: E731
    args = (t["gate"], t["w_post"], t["scale"], t["w_next"], EPS, 1.0)
    a, b = ob.join(irr, t["res"], t["f"], *args), ob.join(irr, turn(t["res"]), turn(t["f"]), *args)
    for k in ("h", "u"):
        np.testing.assert_allclose(turn(a[k][0]), b[k][0], atol=1e-10)


def test_adamw_against_torch_optim():
    import torch
    rng = np.random.default_rng(1)
    p = rng.standard_normal(50)
    tp = torch.from_numpy(p.copy()).requires_grad_()
    opt = torch.optim.AdamW([tp], lr=3e-3, betas=(0.8, 0.95), eps=1e-7, weight_decay=0.05)
    m = v = np.zeros(50)
    for step in range(1, 8):
        g = rng.standard_normal(50)
        tp.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = oo.adamw(p, g, m, v, lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-7, weight_decay=0.05, step=step)
    np.testing.assert_allclose(p, tp.detach().numpy(), rtol=1e-12)


def test_codes_are_the_nearest_and_keep_what_is_not_zero():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(64 * 40) * np.exp(3 * rng.standard_normal(64 * 40))
    for top, signed in ((127, True), (255, False)):
        a = x if signed else np.abs(x)
        q, most = oo.codes(a, top, signed)
        assert np.abs(q).max() == top
        back = oo.values(q, most, top).reshape(-1)
        scale = np.repeat(most, 64)
        # half a code's step in the root of the share of the largest
        root = lambda z: np.sign(z) * np.sqrt(np.abs(z) / scale)  # noqa: E731
        far = np.abs(root(back) - root(a)) * top
        low = np.sqrt(np.abs(a) / scale) * top < 1 if not signed else np.zeros(len(a), bool)
        assert far[~low].max() <= 0.5 + 1e-9 and (signed or np.all(q[a > 0] >= 1))
    z, most = oo.codes(np.zeros(64), 127, True)
    assert not z.any() and not most.any()
