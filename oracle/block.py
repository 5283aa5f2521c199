"""Row norm and block join over irreps rows in float64, forward and backward, from their formulas.

Every function returns {name: (value, size)}: ``size`` is the same expression with every term's
magnitude, what a rounding error of the value is measured against.  ``irreps`` as in oracle.irreps
("MULxLP" terms); a weight or a gate has one entry per channel, shared by its 2l+1 columns.
"""
import numpy as np

from .irreps import parse_irreps


def degrees(irreps):
    """Columns of each channel, in order."""
    return np.array([2 * ir.l + 1 for ir in parse_irreps(irreps) for _ in range(ir.mul)])


def to_columns(c, deg):
    return np.repeat(c, deg, axis=-1)


def to_channels(t, deg):
    return np.add.reduceat(t, np.concatenate([[0], np.cumsum(deg)[:-1]]), axis=-1)


def rstd(x, eps):
    return 1 / np.sqrt((x * x).mean(-1) + eps)


def act(kind, g):
    """(value, derivative)"""
    if kind == "identity":
        return g, np.ones_like(g)
    if kind == "tanh":
        return np.tanh(g), 1 / np.cosh(g) ** 2
    s = 1 / (1 + np.exp(-g))
    ds = 1 / (4 * np.cosh(g / 2) ** 2)
    return (s, ds) if kind == "sigmoid" else (g * s, s + g * ds)


def norm(irreps, x, w, eps):
    deg = degrees(irreps)
    r = rstd(x, eps)
    u = x * r[:, None] * (1 if w is None else to_columns(w, deg))
    return {"u": (u, np.abs(u)), "rstd": (r, r)}


def _through(q, y, r):
    """Gradient through y = x r, r = rstd(x): r (q - y mean(q y)), and its size."""
    r = r[:, None]
    return (r * (q - y * (q * y).mean(-1, keepdims=True)),
            r * (np.abs(q) + np.abs(y) * np.abs(q * y).mean(-1, keepdims=True)))


def norm_grad(irreps, x, w, r, du, add=None):
    deg = degrees(irreps)
    y = x * r[:, None]
    dx, size = _through(du if w is None else du * to_columns(w, deg), y, r)
    if add is not None:
        dx, size = dx + add, size + np.abs(add)
    t = to_channels(du * y, deg)
    return {"grad_x": (dx, size), "grad_w": (t.sum(0), to_channels(np.abs(du * y), deg).sum(0))}


def _factors(irreps, gate, kind, w_post, scale):
    """Per column: the gate's value, the product of scale and post weight; the gate's derivative."""
    deg = degrees(irreps)
    ones = np.ones(len(deg))
    ws = (ones if scale is None else scale) * (ones if w_post is None else w_post)
    if gate is None:
        return deg, 1.0, to_columns(ws, deg), None
    a, da = act(kind, gate)
    return deg, (a if gate.shape[1] == 1 else to_columns(a, deg)), to_columns(ws, deg), da


def join(irreps, res, f, gate, w_post, scale, w_next, eps, alpha, kind="sigmoid", post=True, nxt=True):
    deg, a, ws, _ = _factors(irreps, gate, kind, w_post, scale)
    out, y = {}, f
    if post:
        r = rstd(f, eps)
        out["rstd_f"] = (r, r)
        y = f * r[:, None]
    h = alpha * res + a * ws * y
    size = np.abs(alpha * res) + np.abs(a * ws * y)
    out["h"] = (h, size)
    if nxt:
        r = rstd(h, eps)
        w = 1 if w_next is None else to_columns(w_next, deg)
        # the statistic's error follows the terms' sizes, not their sum's
        spread = np.sqrt((size * size).mean(-1, keepdims=True) * (r * r)[:, None])
        out["u"] = (h * r[:, None] * w, (size + np.abs(h) * spread) * r[:, None] * np.abs(w))
        out["rstd_h"] = (r, r * (1 + spread[:, 0]))
    return out


def join_grad(irreps, dh, du, h, f, gate, w_post, scale, w_next, rstd_f, rstd_h, alpha, kind="sigmoid", post=True,
              nxt=True):
    deg, a, ws, da = _factors(irreps, gate, kind, w_post, scale)
    ones = np.ones(len(deg))
    e, esize = (np.zeros_like(f), np.zeros_like(f)) if dh is None else (dh, np.abs(dh))
    out = {}
    if nxt:
        z = h * rstd_h[:, None]
        g, size = _through(du if w_next is None else du * to_columns(w_next, deg), z, rstd_h)
        e, esize = e + g, esize + size
        out["grad_w_next"] = (to_channels(du * z, deg).sum(0), to_channels(np.abs(du * z), deg).sum(0))
    out["grad_res"] = (alpha * e, np.abs(alpha) * esize)
    y = f * rstd_f[:, None] if post else f
    t, tsize = e * y, esize * np.abs(y)
    if gate is not None:
        # slopes are differences of terms no larger than 1 + |gate|
        loose = 1 + np.abs(gate)
        if gate.shape[1] == 1:
            out["grad_gate"] = (da * (t * ws).sum(-1, keepdims=True),
                                loose * (tsize * np.abs(ws)).sum(-1, keepdims=True))
        else:
            out["grad_gate"] = (da * to_channels(t * ws, deg), loose * to_channels(tsize * np.abs(ws), deg))
    p, psize = to_channels(t * a, deg).sum(0), to_channels(tsize * np.abs(a), deg).sum(0)
    wp, sc = ones if w_post is None else w_post, ones if scale is None else scale
    out["grad_scale"] = (p * wp, psize * np.abs(wp))
    q, qsize = e * a * ws, esize * np.abs(a * ws)
    if post:
        out["grad_w_post"] = (p * sc, psize * np.abs(sc))
        r = rstd_f[:, None]
        out["grad_f"] = (r * (q - y * (q * y).mean(-1, keepdims=True)),
                         r * (qsize + np.abs(y) * (qsize * np.abs(y)).mean(-1, keepdims=True)))
    else:
        out["grad_f"] = (q, qsize)
    return out
