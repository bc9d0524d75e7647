"""The float64 references of the block norm and of clipping (CPU): gradients
against central differences, clipping against its definition."""
import numpy as np
import pytest

from oracle import layer


@pytest.mark.parametrize("gate", [True, False])
def test_block_norm_gradients_are_central_differences(gate):
    rng = np.random.default_rng(3)
    rows, width, eps = 2, 5, 1e-3
    x = {"residual": rng.standard_normal((rows, width)), "y": rng.standard_normal((rows, width)),
         "z": rng.standard_normal((rows, width)), "w_post": rng.uniform(0.5, 1.5, width),
         "res_scale": rng.uniform(-1, 1, width), "w_pre": rng.uniform(0.5, 1.5, width)}
    dx, dn = rng.standard_normal((rows, width)), rng.standard_normal((rows, width))
    if not gate:
        x["z"] = None

    def loss(v):
        out, _ = layer.block_norm_forward(v["residual"], v["y"], v["z"], v["w_post"],
                                          v["res_scale"], v["w_pre"], eps)
        return (out["x"] * dx).sum() + (out["residual"] * dn).sum()

    out, _ = layer.block_norm_forward(*(x[n] for n in ("residual", "y", "z", "w_post", "res_scale",
                                                       "w_pre")), eps)
    g, mag = layer.block_norm_backward(out["residual"], x["y"], x["z"], x["w_post"],
                                       x["res_scale"], x["w_pre"], eps, dx, dn)
    h = 1e-5
    for name in x:
        if x[name] is None:
            continue
        num = np.zeros_like(x[name])
        for at in np.ndindex(num.shape):
            hi, lo = dict(x), dict(x)
            hi[name], lo[name] = x[name].copy(), x[name].copy()
            hi[name][at] += h
            lo[name][at] -= h
            num[at] = (loss(hi) - loss(lo)) / (2 * h)
        d = g["d" + name]
        # h^2 times third derivatives of order 10, and 2^-52 / h
        np.testing.assert_allclose(d, num, rtol=0, atol=1e-8 * max(1, np.abs(d).max()))
        assert (np.abs(d) <= mag["d" + name] * (1 + 1e-12)).all()


def test_clip():
    rng = np.random.default_rng(4)
    g = [rng.standard_normal(n) for n in (1, 7, 0, 30)]
    n, out = layer.clip(g, 0.5, 0.0)
    assert np.isclose(n, np.linalg.norm(np.concatenate(g)))
    assert np.isclose(np.linalg.norm(np.concatenate(out)), 0.5)
    n, out = layer.clip(g, 1e9, 1e-6)
    assert all(np.array_equal(a, b) for a, b in zip(g, out))
    assert layer.clip([np.zeros(3)], 0.0, 0.0)[0] == 0.0
