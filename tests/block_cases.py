"""Cases of the block tests: configurations, seeded inputs, and the bounds on rounding."""
import numpy as np

from oracle import block as ob

EPS = 1e-5
LADDER = "128x0e+128x1o+128x2e+128x3o"
ODD = "19x0e+7x1o+5x2e"

# irreps, rows: one column; a lone channel of several columns; short and odd rows; a degree that comes
# back; rows that end inside a chunk; rows shared by the waves of a workgroup
SHAPES = [("1x0e", 3), ("1x3o", 1), ("4x0e+4x1o", 63), (ODD, 1), (ODD, 517), ("3x0e+2x2e+5x0o", 65),
          ("32x0e+32x1o+32x2e", 130), ("257x0e", 37), ("1031x0e+3x1o", 5), (LADDER, 19)]
DTYPES = ("f32", "f64", "bf16", "f16")
# gate, act, post norm, next norm
CONFIGS = [("channel", "sigmoid", True, True), ("channel", "silu", False, True), ("row", "tanh", True, False),
           ("row", "silu", False, True), (None, "identity", True, True), (None, "identity", False, False),
           ("channel", "identity", True, False), ("channel", "tanh", False, False)]
# wide scalar rows, over waves of one workgroup in every dtype
WIDE = [("4100x0e", 7, "bf16"), ("8192x0e", 1, "f16"), ("2050x0e", 9, "f32"), ("1100x0e", 6, "f64"),
        ("40000x0e", 3, "f32")]
# without a gate per channel: the sums over columns take 144 KB of LDS
BROAD = "9000x0e+9000x1o"
# a degree that changes at every channel: one lane holds a row where the gate is per channel
CHANGING = "+".join(["1x0e+1x1o"] * 20)


def unit(dtype):
    """The larger of a rounding's half steps: of the rows' type, of the arithmetic."""
    return {"f32": 2.0 ** -24, "f64": 2.0 ** -53, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]


def work_unit(dtype):
    return 2.0 ** -53 if dtype == "f64" else 2.0 ** -24


def bound(value, size, dtype, roundings, stored=True):
    """Half a step of the stored type on the value, `roundings` of the arithmetic's on its terms, and
    half the spacing of fp16's subnormal numbers."""
    b = roundings * work_unit(dtype) * size
    if stored:
        b = b + unit(dtype) * np.abs(value) + (2.0 ** -25 if dtype == "f16" else 0.0)
    return b


# Roundings along one result of a row.  A sum over a row is a chain of at most 32 products in a lane
# and a tree of at most ten levels (lanes, then waves): 32 + 10 + 2 for the product and the mean; the
# statistic halves it and adds its root and quotient.  A result holds at most three such sums (the two
# norms' and the gate's), the gate's function (exponential, sum, quotient, product: 8) and a dozen
# products and sums of its own: 3 * 44 + 8 + 12 < 160.
ROW = 160


def weight_roundings(rows):
    """A weight gradient adds its rows to that: at most all of them in a lane's chain (the partial sums
    are added in double), 2l+1 columns and the workgroup's row groups."""
    return ROW + rows + 15 + 256


def inputs(irreps, rows, dtype, config, seed):
    """Row arrays (float64 values that the dtype holds) and weights (float32 or float64)."""
    import torch
    gate, _, post, nxt = config
    rng = np.random.default_rng(seed)
    tdt = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    deg = ob.degrees(irreps)
    c, d = len(deg), int(deg.sum())
    held = lambda a: torch.from_numpy(a).to(tdt)  # noqa: E731
    weight = lambda: torch.from_numpy(1 + 0.2 * rng.standard_normal(c)).to(  # noqa: E731
        torch.float64 if dtype == "f64" else torch.float32)
    f = rng.standard_normal((rows, d)) * np.exp(0.5 * rng.standard_normal((rows, 1)))
    if rows > 2:
        f[rows // 2] = 0  # a receiver without edges
    t = {"x": held(rng.standard_normal((rows, d))), "f": held(f), "res": held(rng.standard_normal((rows, d))),
         "gate": None if gate is None else held(rng.standard_normal((rows, 1 if gate == "row" else c)) * 2),
         "w_post": weight() if post else None, "scale": weight() * 0.5, "w_next": weight() if nxt else None,
         "w": weight(), "du": held(rng.standard_normal((rows, d))), "dh": held(rng.standard_normal((rows, d))),
         "add": held(rng.standard_normal((rows, d)))}
    return t


def wide(t):
    return None if t is None else t.double().numpy()
