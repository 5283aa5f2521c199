"""Group norm over graphs, routing to experts and experts' products over irreps rows in float64, forward
and backward, from their formulas.

Values of sums come as (value, size): ``size`` is the same expression with every term's magnitude, what a
rounding error of the value is measured against.
"""
import numpy as np

from .block import act
from .irreps import parse_irreps


# ------------------------------------------------------------------------------------ group norm

def graphs(ptr):
    return [(int(a), int(b)) for a, b in zip(ptr, ptr[1:])]


def group_stats(x, ptr, groups, eps):
    """(mean, rstd) [graphs][groups]; 0 and eps^(-1/2) for an empty graph."""
    mean, rstd = np.zeros((len(ptr) - 1, groups)), np.full((len(ptr) - 1, groups), eps ** -0.5)
    for s, (a, b) in enumerate(graphs(ptr)):
        if b > a:
            v = x[a:b].reshape(b - a, groups, -1)
            mean[s] = v.mean((0, 2))
            rstd[s] = 1 / np.sqrt(((v - mean[s][:, None]) ** 2).mean((0, 2)) + eps)
    return mean, rstd


def per_row(stat, ptr, rows, channels):
    """A statistic [graphs][groups] for every row and channel; rows of no graph have 0."""
    out = np.zeros((rows, channels))
    for s, (a, b) in enumerate(graphs(ptr)):
        out[a:b] = np.repeat(stat[s], channels // stat.shape[1])
    return out


def group_norm(x, ptr, w, bias, mean, rstd, kind):
    """(y, z): zeros where a row is of no graph."""
    n, c = x.shape
    xh = (x - per_row(mean, ptr, n, c)) * per_row(rstd, ptr, n, c)
    z = xh * w + bias
    inside = np.zeros((n, 1))
    inside[ptr[0]:ptr[-1]] = 1
    return act(kind, z)[0] * inside, z


def group_norm_grad(x, ptr, w, bias, mean, rstd, dy, kind):
    """{name: value}: grad_x, grad_w, grad_bias, and the parts that error bounds are formed from."""
    n, c = x.shape
    g = mean.shape[1]
    r = per_row(rstd, ptr, n, c)
    xh = (x - per_row(mean, ptr, n, c)) * r
    z = xh * w + bias
    inside = np.zeros((n, 1))
    inside[ptr[0]:ptr[-1]] = 1
    slope = act(kind, z)[1]
    dz = dy * slope * inside
    q = dz * w

    def means(t):
        out = np.zeros_like(mean)
        for s, (a, b) in enumerate(graphs(ptr)):
            if b > a:
                out[s] = t[a:b].reshape(b - a, g, -1).mean((0, 2))
        return per_row(out, ptr, n, c)
    dx = r * (q - means(q) - xh * means(q * xh))
    return {"grad_x": dx, "grad_w": (dz * xh).sum(0), "grad_bias": dz.sum(0), "xh": xh, "z": z, "dz": dz, "q": q, "r": r,
            "means": means, "inside": inside}


# ------------------------------------------------------------------------------------ routing

def scores(logits, kind):
    """Scores; a logit of -inf has none."""
    l = np.asarray(logits, dtype=np.float64)
    masked = np.isneginf(l)
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            e = np.where(masked, 0, np.exp(l - l.max(1, keepdims=True)))
            s = e / e.sum(1, keepdims=True)
    return np.where(masked, 0, s)


def shares(l, kind):
    """The chosen logits' scores over their sum: from logarithms, so that scores too small for a double have shares."""
    if not len(l):
        return l
    with np.errstate(all="ignore"):
        t = -np.logaddexp(0, -l) if kind == "sigmoid" else l
        t = np.exp(t - t.max())
        return t / t.sum()


def route(logits, bias, kind, top_k, groups=1, top_groups=1, renormalise=True, scale=1.0):
    """(experts, weights), a row at a time."""
    s = scores(logits, kind)
    n, e = s.shape
    c = s + (0 if bias is None else bias)
    c = np.where(np.isneginf(logits), -np.inf, np.where(np.isnan(c), -np.finfo(np.float64).max, c))
    experts, weights = np.full((n, top_k), -1, np.int32), np.zeros((n, top_k))
    width = e // groups
    for i in range(n):
        keep = np.ones(e, bool)
        if top_groups < groups:
            best = []
            for g in range(groups):
                top = sorted((v for v in c[i, g * width:(g + 1) * width] if v > -np.inf), reverse=True)[:2]
                best.append(sum(top) if top else -np.inf)
            taken = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            keep[:] = False
            for g in taken:
                keep[g * width:(g + 1) * width] = True
        order = sorted((j for j in range(e) if keep[j] and c[i, j] > -np.inf), key=lambda j: (-c[i, j], j))[:top_k]
        p = shares(np.asarray(logits, dtype=np.float64)[i, order], kind) if renormalise else s[i, order]
        experts[i, :len(order)], weights[i, :len(order)] = order, scale * p
    return experts, weights


def route_grad(logits, experts, dp, kind, renormalise=True, scale=1.0):
    """(grad_logits, size)"""
    s = scores(logits, kind)
    out, size = np.zeros_like(s), np.zeros_like(s)
    for i in range(len(s)):
        at = [(int(e), scale * d) for e, d in zip(experts[i], dp[i]) if 0 <= e < s.shape[1]]
        if not at:
            continue
        e, d = np.array([a for a, _ in at]), np.array([b for _, b in at])
        with np.errstate(over="ignore"):
            rest = 1 / (1 + np.exp(logits[i])) if kind == "sigmoid" else 1.0
        if renormalise:
            r = shares(logits[i, e], kind)
            dl, most = r * (d - (d * r).sum()), r * (np.abs(d) + (np.abs(d) * r).sum())
        else:
            dl, most = d * s[i, e], np.abs(d) * s[i, e]
        np.add.at(out[i], e, dl)
        np.add.at(size[i], e, most)
        out[i], size[i] = out[i] * rest, size[i] * rest
        if kind == "softmax" and not renormalise:  # every logit has a part in the chosen scores
            out[i] -= s[i] * dl.sum()
            size[i] += s[i] * most.sum()
    return out, size


def order(experts, e):
    """(rows, slots, offsets), by sorting."""
    n, k = experts.shape
    ok = np.where((experts >= 0) & (experts < e), experts, e).astype(np.int64)
    flat = ok.reshape(-1)
    slots = np.argsort(flat, kind="stable")
    offsets = np.array([(flat < i).sum() for i in range(e + 1)])
    if k == 1:
        key = ok[:, 0]
    else:
        low = np.sort(ok, axis=1)
        bins = min(e, 4096 // e)
        b = np.where(low[:, 1] == e, low[:, 0], low[:, 1])
        key = np.where(low[:, 0] == e, e * bins, low[:, 0] * bins + b * bins // e)
    return np.argsort(key, kind="stable").astype(np.int32), slots.astype(np.int32), offsets.astype(np.int32)


# ------------------------------------------------------------------------------------ experts' products

def paths(in_irreps, out_irreps):
    """[(mul_in, first column, mul_out, first column, 2l+1, first weight)], weights, columns in, columns out."""
    def columns(text):
        got, at = [], 0
        for ir in parse_irreps(text):
            got.append((ir, at))
            at += ir.mul * (2 * ir.l + 1)
        return got, at
    (ins, d_in), (outs, d_out) = columns(in_irreps), columns(out_irreps)
    found, at = [], 0
    for a, xa in ins:
        for b, ya in outs:
            if a.l == b.l and a.p == b.p:
                found.append((a.mul, xa, b.mul, ya, 2 * a.l + 1, at))
                at += a.mul * b.mul
    return found, at, d_in, d_out


def dense(in_irreps, out_irreps, w):
    """The matrix [d_out][d_in] of one expert's weights."""
    found, _, d_in, d_out = paths(in_irreps, out_irreps)
    m = np.zeros((d_out, d_in))
    for mi, xa, mo, ya, k, at in found:
        block = w[at:at + mi * mo].reshape(mo, mi)
        for i in range(k):
            m[ya + i:ya + mo * k:k, xa + i:xa + mi * k:k] += block
    return m


def linear(in_irreps, out_irreps, x, w, experts=None, weights=None, grad_out=None):
    """{name: (value, size)}: out, and with grad_out grad_x, grad_w and grad_weights."""
    found, numel, d_in, d_out = paths(in_irreps, out_irreps)
    n, e = len(x), len(w)
    if experts is None:
        experts, weights = np.zeros((n, 1), int), np.ones((n, 1))
    k = experts.shape[1]
    out = {"out": [np.zeros((n, d_out)), np.zeros((n, d_out))]}
    if grad_out is not None:
        out.update(grad_x=[np.zeros((n, d_in)), np.zeros((n, d_in))], grad_w=[np.zeros((e, numel)), np.zeros((e, numel))],
                   grad_weights=[np.zeros((n, k)), np.zeros((n, k))])
    for i in range(e):
        row, j = np.nonzero(experts == i)
        if not len(row):
            continue
        m = dense(in_irreps, out_irreps, w[i])
        for s, f in ((0, lambda t: t), (1, np.abs)):
            p, xi, mi = f(weights[row, j])[:, None], f(x[row]), f(m)
            np.add.at(out["out"][s], row, p * (xi @ mi.T))
            if grad_out is None:
                continue
            g = f(grad_out[row])
            back = g @ mi
            np.add.at(out["grad_x"][s], row, p * back)
            out["grad_weights"][s][row, j] = (back * xi).sum(1)
            for a, xa, b, ya, c, at in found:
                gi, xs = (g * p)[:, ya:ya + b * c].reshape(-1, b, c), xi[:, xa:xa + a * c].reshape(-1, a, c)
                out["grad_w"][s][i, at:at + a * b] = np.einsum("nvm,num->vu", gi, xs).reshape(-1)
    return {name: tuple(v) for name, v in out.items()}
