"""Float64 references of the norms around a block and of gradient clipping
(test infrastructure), from their definitions; the block norm's come with the
sums of the terms' magnitudes (the scale that rounding errors go by)."""
import numpy as np


def _silu(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s, s * (1.0 + z * (1.0 - s))


def block_norm_forward(residual, y, z, w_post, res_scale, w_pre, eps):
    """{"residual", "x"} and their magnitudes"""
    al = np.ones_like(w_post) if res_scale is None else res_scale
    iy = 1.0 / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps)
    u = y * iy * w_post * (1.0 if z is None else _silu(z)[0])
    new = residual + al * u
    ir = 1.0 / np.sqrt((new ** 2).mean(-1, keepdims=True) + eps)
    m = np.abs(residual) + np.abs(al * u)
    mi = ir * (1.0 + ir ** 2 * (np.abs(new) * m).mean(-1, keepdims=True))
    return ({"residual": new, "x": new * ir * w_pre},
            {"residual": m, "x": np.abs(w_pre) * m * mi})


def block_norm_backward(new, y, z, w_post, res_scale, w_pre, eps, dx, dnew=None, stats=None):
    """stats: (inv_y, inv_r) [rows][1] in place of those of y and new"""
    al = np.ones_like(w_post) if res_scale is None else res_scale
    width = y.shape[-1]
    mean = lambda a: a.sum(-1, keepdims=True) / width  # noqa: E731
    iy, ir = stats or (1.0 / np.sqrt(mean(y ** 2) + eps), 1.0 / np.sqrt(mean(new ** 2) + eps))
    s, ds = (np.ones_like(y), np.zeros_like(y)) if z is None else _silu(z)
    # magnitudes of silu' (its two terms may cancel)
    ms = np.zeros_like(y) if z is None else (1.0 + np.abs(z)) / (1.0 + np.exp(-z))
    t = dx * w_pre
    dr = ir * t - new * ir ** 3 * mean(t * new)
    mdr = np.abs(ir * t) + np.abs(new) * ir ** 3 * mean(np.abs(t * new))
    if dnew is not None:
        dr, mdr = dr + dnew, mdr + np.abs(dnew)
    n = y * iy
    q, mq = al * dr * s * w_post, np.abs(al * s * w_post) * mdr
    out = {"dresidual": dr, "dy": q * iy - y * iy ** 3 * mean(q * y),
           "dz": None if z is None else al * dr * n * w_post * ds,
           "dw_post": (al * dr * n * s).sum(0),
           "dres_scale": None if res_scale is None else (dr * n * w_post * s).sum(0),
           "dw_pre": (dx * new * ir).sum(0)}
    mag = {"dresidual": mdr, "dy": mq * iy + np.abs(y) * iy ** 3 * mean(mq * np.abs(y)),
           "dz": None if z is None else np.abs(al * n * w_post) * mdr * ms,
           "dw_post": (np.abs(al * n * s) * mdr).sum(0),
           "dres_scale": None if res_scale is None else (np.abs(n * w_post * s) * mdr).sum(0),
           "dw_pre": np.abs(dx * new * ir).sum(0)}
    return out, mag


def clip(grads, max_norm, eps):
    """(norm, the scaled gradients)"""
    n = np.sqrt(sum((np.asarray(g, dtype=np.float64) ** 2).sum() for g in grads))
    c = min(1.0, max_norm / (n + eps)) if n + eps else 1.0
    return n, [g * c for g in grads]
