"""Routing to experts on the GPU against the float64 oracle: choices exactly, weights and gradients within counted
roundings; ties, masks, values that are not finite, the lists, streams and graphs."""
import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import experts as ox

from block_cases import work_unit
from expert_cases import DTYPES, held, host, real, within

pytestmark = pytest.mark.gpu

# experts, top_k, groups, top_groups, rows: one expert; one lane; odd counts; several lanes; groups of one, of a part of
# a lane and of several lanes; as many choices as experts; a whole wave to a row
SHAPES = [(1, 1, 1, 1, 5), (3, 2, 1, 1, 1), (8, 2, 1, 1, 1000), (17, 5, 1, 1, 77), (64, 6, 8, 4, 333), (40, 4, 5, 2, 65),
          (6, 3, 6, 3, 130), (96, 8, 3, 2, 50), (8, 8, 1, 1, 64), (200, 32, 1, 1, 41), (512, 4, 1, 1, 30),
          (256, 8, 8, 4, 60), (512, 3, 64, 5, 20), (33, 2, 33, 9, 21)]


def up(a, device):
    import torch
    return (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).to(device)


def inputs(n, e, k, dtype, seed, masked=0.15):
    rng = np.random.default_rng(seed)
    l = 2 * rng.standard_normal((n, e)) + rng.standard_normal(e)
    l[rng.random((n, e)) < masked] = -np.inf
    if n > 3:
        l[n // 3] = -np.inf
        l[n // 2] = -30000.0
    return held(l, dtype), real(0.2 * rng.standard_normal(e), dtype), real(rng.standard_normal((n, k)), dtype)


def weight_bound(p, dtype, e, k):
    """The stored type's half step, and in double the exponentials, the two sums and a dozen operations (an argument's
    rounding times its size, below 750, is in each exponential)."""
    return (2.0 ** -24 if dtype != "f64" else 0) * np.abs(p) + (2 * 750 + e + k + 16) * 2.0 ** -53 * np.abs(p) + 1e-300


def grad_bound(logits, size, dtype, e, k):
    """Every share comes of an exponential of a difference, whose rounding its size multiplies, of sums of e or k terms,
    and of a dozen operations; the gradient's terms hold two shares.  What underflows counts as the smallest normal."""
    u = work_unit(dtype)
    finite = np.where(np.isfinite(logits), logits, 0)
    span = (finite.max(1) - finite.min(1) + np.abs(finite).max(1))[:, None]
    return 2 * u * (np.minimum(span, 800) + e + k + 16) * size + (1e-37 if dtype != "f64" else 1e-300)


def check(router, logits, bias, dp, device, dtype):
    n, k, e = logits.shape[0], router.top_k, router.experts
    l = host(logits)
    d = up(logits, device)
    kw = dict(renormalise=router.renormalise, scale=router.scale)
    experts, weights = cg.route_forward(router, d, None if bias is None else up(bias, device))
    want, p = ox.route(l, None if bias is None else host(bias), router.score, k, router.groups, router.top_groups, **kw)
    assert np.array_equal(experts.cpu().numpy(), want)
    within("weights", weights, p, weight_bound(p, dtype, e, k))
    got = cg.route_backward(router, d, experts, up(dp, device))
    value, size = ox.route_grad(l, want, host(dp), router.score, **kw)
    within("grad_logits", got, value, grad_bound(l, size, dtype, e, k), dtype)
    order = cg.route_order(router, experts)
    for name, a, b in zip(order._fields, order, ox.order(want, e)):
        assert np.array_equal(a.cpu().numpy(), b), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e, k, groups, top_groups, n", SHAPES)
def test_shapes(device, e, k, groups, top_groups, n, score, dtype):
    logits, bias, dp = inputs(n, e, k, dtype, 31)
    for renorm in (True, False):
        router = cg.router_for(e, k, dtype, score=score, groups=groups, top_groups=top_groups, renormalise=renorm, scale=1.5)
        check(router, logits, bias if renorm else None, dp, device, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest(device, score, dtype):
    """Equal logits everywhere, in runs, and scores that saturate; equal groups too."""
    rng = np.random.default_rng(32)
    l = np.round(rng.standard_normal((400, 24)))
    l[0], l[1, ::2], l[2] = 0, 3, 60 + np.arange(24)  # sigmoid: 1 for every one
    for groups, top in ((1, 1), (4, 2), (8, 3)):
        router = cg.router_for(24, 3, dtype, score=score, groups=groups, top_groups=top)
        check(router, held(l, dtype), None, real(np.ones((400, 3)), dtype), device, dtype)


def test_neighbouring_scores_are_told_apart(device):
    """Logits one step of float apart, at scores where float's own sigmoid and softmax give one value."""
    l = np.full((64, 8), 12.0, np.float32)
    for i in range(64):
        l[i, i % 8] = np.nextafter(np.float32(12), np.float32(13))
        l[i, (i + 3) % 8] = np.nextafter(np.float32(12), np.float32(11))
    for score in ("softmax", "sigmoid"):
        experts, _ = cg.route_forward(cg.router_for(8, 8, "f32", score=score), up(l, device))
        e = experts.cpu().numpy()
        assert np.array_equal(e[:, 0], np.arange(64) % 8) and np.array_equal(e[:, 7], (np.arange(64) + 3) % 8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_are_not_finite(device, score):
    """The lowest value of the type is no mask; -inf in logits or bias is; a row's NaN or inf stays in its row."""
    import torch
    lowest = float(np.finfo(np.float32).min)
    l = torch.randn(6, 5, generator=torch.Generator().manual_seed(3))
    l[0, 1:] = lowest
    l[1, 2] = float("nan")
    l[2, 3] = float("inf")
    l[3, :] = float("nan")
    router = cg.router_for(5, 3, "f32", score=score, renormalise=False)
    experts, weights = cg.route_forward(router, l.to(device))
    e, p = experts.cpu().numpy(), weights.cpu().numpy()
    assert e[0].tolist() == [0, 1, 2] and p[0, 1] == 0 and p[0, 2] == 0
    assert ((0 <= e) & (e < 5)).all() and all(len(set(r)) == 3 for r in e.tolist())
    if score == "softmax":
        assert np.isnan(p[1:4]).all()
    else:
        assert np.isfinite(p[1]).all() and 2 not in e[1] and e[2, 0] == 3 and p[2, 0] == 1 and np.isnan(p[3]).all()
    assert np.isfinite(p[4:]).all()
    bias = torch.zeros(5)
    bias[torch.tensor([0, 2, 4])] = float("-inf")
    experts, weights = cg.route_forward(router, l[4:].to(device), bias.to(device))
    assert (experts[:, 2] == -1).all() and (weights[:, 2] == 0).all()
    assert set(experts[:, :2].flatten().tolist()) == {1, 3}


def test_pitch_and_given_outputs(device):
    import torch
    router = cg.router_for(12, 2, "bf16", score="sigmoid")
    wide = torch.randn(100, 31, device=device).bfloat16()
    logits = wide[:, 5:17]
    want = cg.route_forward(router, logits.contiguous())
    e, p = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = cg.route_forward(router, logits, experts=e, weights=p)
    assert got[0] is e and e.equal(want[0]) and p.equal(want[1])
    assert cg.route_backward(router, logits, e, p).equal(cg.route_backward(router, logits.contiguous(), e, p))


def test_backward_skips_experts_out_of_range(device):
    import torch
    router = cg.router_for(6, 3, "f32", score="sigmoid", renormalise=False)
    l = torch.randn(4, 6, device=device)
    e = torch.tensor([[0, -1, 5], [6, 2, 1 << 30], [-5, -1, -1], [3, 3, 1]], dtype=torch.int32, device=device)
    got = cg.route_backward(router, l, e, torch.ones(4, 3, device=device))
    s = torch.sigmoid(l.double())
    want = torch.zeros_like(s)
    for i, j, times in ((0, 0, 1), (0, 5, 1), (1, 2, 1), (3, 3, 2), (3, 1, 1)):
        want[i, j] = times * s[i, j] * (1 - s[i, j])
    assert torch.allclose(got.double(), want, rtol=1e-6, atol=1e-7)


# ------------------------------------------------------------------------------------ lists

# rows, top_k, experts: nothing; one workgroup; its last size; several waves, many keys, everything on one expert
@pytest.mark.parametrize("n, k, e", [(0, 2, 4), (1, 1, 1), (5, 3, 512), (1000, 2, 64), (8192, 2, 7), (8193, 2, 7), (16385, 1, 300),
                                     (70_001, 4, 16), (200_003, 6, 64), (30_000, 2, 512), (100_000, 1, 1)])
def test_lists(device, n, k, e):
    import torch
    rng = np.random.default_rng(n + k)
    experts = np.minimum(rng.integers(0, e, (n, k)), rng.integers(0, e, (n, k))).astype(np.int32)
    experts[rng.random((n, k)) < 0.1] = -1
    experts[rng.random((n, k)) < 0.02] = e + 3
    experts[rng.random((n, k)) < 0.01] = np.iinfo(np.int32).min
    experts[rng.random((n, k)) < 0.01] = np.iinfo(np.int32).max
    router = cg.router_for(max(e, k), k, "f32")
    e = router.experts
    got = cg.route_order(router, up(experts, device))
    for name, a, b in zip(got._fields, got, ox.order(experts, e) if n else (np.zeros(0), np.zeros(0), np.zeros(e + 1))):
        assert np.array_equal(a.cpu().numpy(), b), name
    again = cg.route_order(router, up(experts, device))
    assert all(a.equal(b) for a, b in zip(got, again))


def test_streams_and_graphs(device):
    """Another stream, and two captured graphs replayed in turn on changing logits, against eager calls."""
    import torch
    router = cg.router_for(32, 4, "f32", score="sigmoid", groups=4, top_groups=2)
    logits = [torch.randn(n, 32, device=device) for n in (500, 20_000)]

    def run(l, stream=None):
        experts, weights = cg.route_forward(router, l, stream=stream)
        return (experts, weights) + tuple(cg.route_order(router, experts, stream=stream)) + \
            (cg.route_backward(router, l, experts, weights, stream=stream),)
    want = [run(l) for l in logits]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [run(l, side) for l in logits]
    torch.cuda.current_stream().wait_stream(side)
    assert all(a.equal(b) for w, g in zip(want, got) for a, b in zip(w, g))
    graphs, outs = [], []
    torch.cuda.synchronize()
    for l in logits:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(l))
    for i in range(3):
        for l in logits:
            l.copy_(torch.randn(l.shape, device=device))
        for g in graphs:
            g.replay()
        for l, o in zip(logits, outs):
            assert all(a.equal(b) for a, b in zip([t.clone() for t in o], run(l))), i
