"""AdamW over flat arrays: the formula in float64, and the 8-bit codes of its moments.

``codes`` and ``values`` follow the definition operation by operation in the arrays' own precision:
in float32 they give the code that a float32 implementation has to give, in float64 the definition's.
"""
import numpy as np

BLOCK = 64


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, factor=1.0):
    """(p, m, v) after one step."""
    g = g * factor
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mhat, vhat = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * (mhat / (np.sqrt(vhat) + eps) + weight_decay * p), m, v


def clip_factor(norm, max_norm, grad_scale=1.0):
    n = abs(grad_scale) * norm
    return grad_scale * (max_norm / n if max_norm > 0 and n > max_norm else 1.0)


def codes(x, top, signed):
    """(codes, scales) of an array of whole blocks; NaN and codes of 0 for a block with a value that is
    not finite."""
    f = x.dtype.type
    a = np.abs(x).reshape(-1, BLOCK)
    finite = np.isfinite(a).all(1)
    a = np.where(finite[:, None], a, f(0))
    most = a.max(1)
    most = np.where(most < np.finfo(np.float32).tiny, f(0), most)
    inv = np.where(most > 0, f(1) / np.where(most > 0, most, f(1)), f(0))
    q = np.rint(np.sqrt(a * inv[:, None]) * f(top))
    if not signed:
        q = np.where((a > 0) & (most > 0)[:, None], np.maximum(q, f(1)), q)
    q = q.reshape(-1)
    return (np.where(x < 0, -q, q) if signed else q).astype(np.int32), np.where(finite, most, f(np.nan))


def values(q, most, top):
    f = most.dtype.type
    t = q.astype(f) * f(1.0 / top)
    return (t * np.abs(t)).reshape(-1, BLOCK) * most[:, None]
