"""Cases of the group norm, routing and experts' tests: seeded inputs, and the bounds on rounding."""
import re

import numpy as np

from oracle import experts as ox

from block_cases import unit, work_unit

DTYPES = ("f32", "f64", "bf16", "f16")


def torch_type(dtype):
    import torch
    return {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def held(a, dtype):
    """A tensor of values that the dtype holds."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch_type(dtype))


def real(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.float64 if dtype == "f64" else torch.float32)


def host(t):
    return t.detach().double().cpu().numpy()


def within(name, got, value, most, dtype=None):
    """|got - value| within `most`, half a step of the stored type on top (dtype None: not stored in it)."""
    got = host(got).reshape(value.shape)
    if dtype is not None:
        most = most + unit(dtype) * (np.abs(value) + most) + (2.0 ** -25 if dtype == "f16" else 0.0)
    off = np.abs(got - value)
    assert np.all(off <= most), f"{name}: {np.nanmax(off / np.maximum(most, 1e-300)):.3g} of the bound, " \
                                f"{int(np.isnan(off).sum())} not numbers"


# ------------------------------------------------------------------------------------ group norm

# channels, groups, graphs' sizes: one channel; one row; empty graphs; groups inside a lane's channels and over
# many lanes; odd rows; several slots of a lane; as many groups as channels; graphs of one workgroup beside graphs over
# many, and these over as many chunks as there are
NORM_SHAPES = [(1, 1, [3]), (4, 2, [1]), (4, 4, [0, 5, 0, 0, 9, 0]), (32, 4, [21] * 24), (95, 5, [700, 1, 3, 0, 411]),
               (64, 64, [130, 2]), (2048, 4, [9, 30]), (513, 3, [40]), (24, 1, [1, 1, 1, 2]), (130, 13, [900]),
               (16, 16, [5000, 1, 7000]), (40, 8, [1] * 300 + [9000, 4, 2600, 0] + [7] * 300), (1024, 512, [3000, 20]),
               (2047, 1, [70, 3])]


def norm_inputs(channels, graphs, dtype, seed, outside=(2, 3)):
    """x, w, bias, dy and ptr, with rows of no graph around them."""
    rng = np.random.default_rng(seed)
    n = sum(graphs) + sum(outside)
    ptr = np.concatenate([[0], np.cumsum(graphs)]) + outside[0]
    x = rng.standard_normal((n, channels)) * np.exp(0.3 * rng.standard_normal(channels)) + 2 * rng.standard_normal(channels)
    return {"x": held(x, dtype), "dy": held(rng.standard_normal((n, channels)), dtype),
            "w": real(1 + 0.2 * rng.standard_normal(channels), dtype), "bias": real(0.3 * rng.standard_normal(channels), dtype),
            "ptr": ptr.astype(np.int32)}


def norm_roundings(norm, rows):
    """Additions that one result of a sum over rows x channels passes through.  In a lane: the 64 rows at most that it holds,
    and its channels of a group; or along a chunk, a 1,024th of the rows at least, its batches of rows, each joined in 4
    roundings after 5 of its own.  Over a workgroup: a group's sums of RG rows by threads / GP threads (one, of fewer threads
    than groups), a tree of 6 and up to 16 waves.  Over a graph's pieces: 256 threads or more join them, GP side by side, in 4
    roundings each, then a tree of 10 joins.  A dozen products and quotients."""
    c = {m[0]: int(m[1]) for m in re.findall(r"constexpr int (\w+) = (\d+);", norm.source)}
    step = c["RW"] * (4 if c["NS"] * c["CV"] <= 4 else 2)
    batches = -(-rows // (1024 * step))
    pieces = rows // (batches * step) + 1
    lanes = c["RW"] * c["W"] * c["GP"] // 64 + min(16, c["GP"] // 64) * c["RW"] * c["W"] + 1
    return 64 + c["CV"] + 9 * batches + lanes + 6 + 16 + 4 * (min(pieces, 1024) * c["GP"] // 256 + 1) + 40 + 12


def stat_bounds(x, ptr, mean, rstd, u, c):
    """Bounds on mean and rstd.  A mean is off by c roundings of the largest |x|.  Squared distances are taken
    from a batch's own mean or joined from differences of means, so each is off by the product of a distance with that
    error, and by its square; their sum passes c roundings.  rstd = (v + eps)^(-1/2) multiplies v's by rstd^3 / 2."""
    dm, dr = np.zeros_like(mean), np.zeros_like(rstd)
    for s, (a, b) in enumerate(ox.graphs(ptr)):
        if b == a:
            dr[s] = 4 * u * rstd[s]
            continue
        v = x[a:b].reshape(b - a, mean.shape[1], -1)
        most, var = np.abs(v).max((0, 2)), v.var((0, 2))
        dm[s] = c * u * most
        dvar = c * u * var + 2 * np.sqrt(var) * dm[s] + dm[s] ** 2
        dr[s] = 0.5 * rstd[s] ** 3 * dvar * (1 + 1e-3) + 4 * u * rstd[s]
    return dm, dr


# The activation's derivative is at most 1.1 and its second derivative at most 1; the function's own error
# is within 16 roundings of (|z| + 1) (16-bit types: the hardware's exponential and reciprocal, |z| 2^-23 and 2^-23).
def act_error(z, dz, u):
    return 1.1 * dz + 16 * u * (np.abs(z) + 1)


# ------------------------------------------------------------------------------------ experts' products

# irreps in, out, experts, top_k, rows: one value; every block size around 16; odd ones; an irrep twice on both
# sides, one without a pair; high degrees; wide blocks in several units; more experts than rows; a plain layer; most experts
# of a row; an irrep that fills LDS
LINEAR_CASES = [("1x0e", "1x0e", 1, 1, 1), ("4x0e+4x1o", "4x1o+4x0e", 3, 2, 15), ("16x1o", "16x1o", 4, 1, 16),
                ("17x0e+33x1o+5x2e", "33x0e+15x1o+7x2e", 5, 3, 67), ("8x0e+4x0e+3x1o", "5x0e+6x0e+2x1o+3x2e", 2, 2, 130),
                ("3x7o+2x4e+40x3o", "2x7o+40x3o+5x4e", 3, 2, 33), ("128x0e+100x2e", "130x0e+65x2e", 6, 2, 50),
                ("64x0e+64x1o", "64x0e+64x1o", 64, 2, 9), ("48x0e+20x1e", "31x0e+20x1e", 1, 0, 1030),
                ("32x0e+32x1o+32x2e", "32x0e+32x1o+32x2e", 8, 2, 700), ("5x1e", "3x1e", 9, 8, 40),
                ("200x0e", "7x0e", 4, 4, 513),
                ("9x0e+3x1o", "3x1o+9x0e", 40, 32, 60), ("390x1o", "40x1o+3x0e", 2, 1, 40)]


def linear_inputs(a, b, e, k, n, dtype, seed, free=True):
    """Inputs; a tenth of the slots and some whole rows without an expert (free), one row naming an expert twice."""
    rng = np.random.default_rng(seed)
    _, numel, d_in, d_out = ox.paths(a, b)
    t = {"x": held(rng.standard_normal((n, d_in)), dtype), "w": held(rng.standard_normal((e, numel)) / 4, dtype),
         "g": held(rng.standard_normal((n, d_out)), dtype), "experts": None, "weights": None}
    if k:
        experts = np.argsort(rng.standard_normal((n, e)) + rng.standard_normal(e), axis=1)[:, :k].astype(np.int32)
        if free:
            experts[rng.random((n, k)) < 0.1] = -1
            experts[rng.random(n) < 0.05] = -1
            if k > 1 and n > 2:
                experts[n // 2, :2] = 0
        t["experts"], t["weights"] = experts, real(rng.standard_normal((n, k)), dtype)
    return t


def linear_bounds(a, b, dtype, k, slots):
    """Roundings of (out, grad_x, grad_weights, grad_w) relative to the sums of their terms' sizes.  A matrix
    instruction may truncate where it adds, up to twice a rounding, and every term passes at most as many additions as
    its sum has terms: twice the channels of every pair and a product each, then the weight's product and sum for
    each of k experts (3).  grad_weights adds a dot product over the row to grad_x's, shared by units, lanes and waves.
    grad_w sums an expert's slots and 2l+1 components, with the product p g and the stretches' sums in double."""
    found, _, d_in, d_out = ox.paths(a, b)
    ins, outs = sum(p[0] for p in found), sum(p[2] for p in found)
    u = work_unit(dtype)
    most = max(p[4] for p in found)
    fwd, bwd = 2 * ins + 3 * k + 4, 2 * outs + 3 * k + 4
    return fwd * u, bwd * u, (bwd + d_in + 8) * u, (2 * slots * most + 8) * u + (unit(dtype) if dtype in ("bf16", "f16") and k else 0)
