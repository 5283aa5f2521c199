"""The oracle of group norm, routing and experts' products against differences of its own forward."""
import numpy as np
import pytest

from oracle import experts as ox

H = 1e-6


def differences(f, x, g):
    """d/dx of sum(g * f(x)) by central differences."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        out[i] = ((f(a) - f(b)) * g).sum() / (2 * H)
    return out


# central differences of step 1e-6: truncation h^2 f''' / 6 and cancellation 2^-53 |f| / h, both below 1e-8 here
CLOSE = dict(rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("kind", ["identity", "sigmoid", "silu", "tanh"])
def test_group_norm_gradients(kind):
    rng = np.random.default_rng(1)
    x, w, b, dy = rng.standard_normal((7, 4)), 1 + rng.standard_normal(4), rng.standard_normal(4), rng.standard_normal((7, 4))
    ptr, eps = np.array([1, 4, 4, 6]), 0.1

    def y(x, w, b):
        return ox.group_norm(x, ptr, w, b, *ox.group_stats(x, ptr, 2, eps), kind)[0]
    got = ox.group_norm_grad(x, ptr, w, b, *ox.group_stats(x, ptr, 2, eps), dy, kind)
    np.testing.assert_allclose(got["grad_x"], differences(lambda t: y(t, w, b), x, dy), **CLOSE)
    np.testing.assert_allclose(got["grad_w"], differences(lambda t: y(x, t, b), w, dy), **CLOSE)
    np.testing.assert_allclose(got["grad_bias"], differences(lambda t: y(x, w, t), b, dy), **CLOSE)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_gradients(kind, renorm):
    rng = np.random.default_rng(2)
    l, dp = rng.standard_normal((5, 6)), rng.standard_normal((5, 3))
    l[0, 1] = -np.inf
    experts, _ = ox.route(l, None, kind, 3, renormalise=renorm, scale=1.5)

    def weights(t):
        s = ox.scores(t, kind)
        p = np.take_along_axis(s, experts, 1)
        return 1.5 * (p / p.sum(1, keepdims=True) if renorm else p)
    with np.errstate(invalid="ignore"):
        want = differences(weights, l, dp)
    want[0, 1] = 0
    np.testing.assert_allclose(ox.route_grad(l, experts, dp, kind, renorm, 1.5)[0], want, **CLOSE)


def test_route_choice():
    l = np.array([[0.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [1.0, -np.inf, -np.inf, -np.inf]])
    experts, weights = ox.route(l, None, "sigmoid", 2)
    assert experts.tolist() == [[1, 2], [-1, -1], [0, -1]]
    assert weights.tolist() == [[0.5, 0.5], [0, 0], [1, 0]]
    # groups {0, 1}, {2, 3}: sums of 2 and 1.5 of the logits' scores; the best expert lies in the other one
    l = np.log(np.array([[1.0, 1.0, 1.6, 0.1]]))
    assert ox.route(l, None, "softmax", 2, groups=2, top_groups=1)[0].tolist() == [[0, 1]]
    rows, slots, offsets = ox.order(np.array([[2, 0], [1, 0], [-1, 2], [0, 1]], np.int32), 3)
    assert rows.tolist() == [1, 3, 0, 2] and slots.tolist() == [1, 3, 6, 2, 7, 0, 5, 4] and offsets.tolist() == [0, 3, 5, 7]


def test_linear_gradients_and_rotation():
    rng = np.random.default_rng(3)
    a, b = "2x0e+3x1o+1x0e", "2x1o+2x0e+1x2e"
    numel, d_in, d_out = ox.paths(a, b)[1:]
    assert (numel, d_in, d_out) == (2 * 2 + 3 * 2 + 1 * 2, 12, 13)
    x, w, p, g = rng.standard_normal((4, d_in)), rng.standard_normal((3, numel)), rng.random((4, 2)), rng.standard_normal((4, d_out))
    e = np.array([[0, 2], [1, 0], [2, -1], [1, 1]])

    def out(x, w, p):
        return ox.linear(a, b, x, w, e, p)["out"][0]
    got = ox.linear(a, b, x, w, e, p, g)
    np.testing.assert_allclose(got["grad_x"][0], differences(lambda t: out(t, w, p), x, g), **CLOSE)
    np.testing.assert_allclose(got["grad_w"][0], differences(lambda t: out(x, t, p), w, g), **CLOSE)
    np.testing.assert_allclose(got["grad_weights"][0], differences(lambda t: out(x, w, t), p, g), **CLOSE)
    assert not got["out"][0][:, 8:].any()               # 2e has no pair
    # a rotation of the vectors' components passes through
    turn = np.linalg.qr(rng.standard_normal((3, 3)))[0]
    y = x.copy()
    y[:, 2:11] = (x[:, 2:11].reshape(-1, 3, 3) @ turn).reshape(-1, 9)
    turned = out(y, w, p)
    np.testing.assert_allclose(turned[:, :6], (out(x, w, p)[:, :6].reshape(-1, 2, 3) @ turn).reshape(-1, 6), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(turned[:, 6:8], out(x, w, p)[:, 6:8], rtol=1e-12, atol=1e-12)
