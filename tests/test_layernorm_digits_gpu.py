"""Layer norm of rows whose mean is large against their spread.

Tolerance.  A warp takes its columns' mean off, the rest's own mean is found from the
differences (exact where an element is within a factor of two of the mean) and taken off
too.  So n is off by what a sum of differences is: a tree of at most 40 roundings of
2^-24 of mean |x - mean|, times inv, and 40 * 2^-24 of n; y by that times w, its own
rounding and the bias's: 2^-24 each.  The mean's rounding, 2^-24 of the mean, is not in
it."""
import numpy as np
import pytest

from test_parity_layernorm_gpu import EPS, U, _built, dev, host, inputs, stats  # noqa: F401

pytestmark = pytest.mark.gpu
# rows, width: one warp a row and several, in both rules of the forward, unaligned rows
SHAPES = [(1, 250), (40, 768), (5000, 768), (700, 2048), (9, 4096), (2, 8192), (33, 1537), (3000, 513),
          (800, 5000)]


@pytest.mark.parametrize("value", [100.3, 1000.1, -3.3e7, 1e30])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_constant_rows(rows, width, value):
    """Every element of a constant row is its mean, and y the bias.  A sum of equal terms
    is off by 20 * 2^-24 of itself at most (its tree), what is left of an element is that
    small, and its own mean is found to 40 * 2^-24 of it: n is within 800 * 2^-48 |value|
    inv, and inv = 1 / sqrt(eps) or less."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    x = torch.full((rows, width), value, device="cuda")
    b = torch.randn(width, device="cuda")
    y, st = ssd.layer_norm_forward(x, None, b, EPS)
    off = 800 * U * U * abs(value) / EPS ** 0.5
    assert (np.abs(host(y) - host(b)) <= off + U * np.abs(host(b))).all()
    assert torch.equal(st[:, 0], x[:, 0])
    g = ssd.layer_norm_backward(x, None, torch.ones_like(x), EPS)
    assert (np.abs(host(g["dweight"])) <= 2 * rows * off).all()


@pytest.mark.parametrize("offset", [4096.0, 1e5])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_a_large_mean(rows, width, offset):
    import state_space_model_analytic_gb300 as ssd
    i = inputs(rows, width, "f32", 5, offset)
    x, w, b = i["x"], i["w"], i["b"]
    mean, inv = stats(x, EPS)
    n = (x - mean) * inv
    ref = n * w + b
    dn = 40 * np.abs(n) + 40 * np.abs(n).mean(-1, keepdims=True)
    y, st = ssd.layer_norm_forward(dev(x), dev(w), dev(b), EPS)
    most = U * (dn * np.abs(w) + 2 * np.abs(b) + 2 * np.abs(ref)) + 1e-30
    err = np.abs(host(y) - ref)
    assert (err <= most).all(), float((err / most).max())
    # the statistics: the mean to its own rounding, inv to that of a sum of squares
    assert (np.abs(host(st)[:, :1] - mean) <= U * (np.abs(mean) + 40 / inv)).all()
    assert (np.abs(host(st)[:, 1:] - inv) <= 40 * U * inv).all()
    # without statistics the gradients have the same n
    dy = i["dy"]
    g = ssd.layer_norm_backward(dev(x), dev(w), dev(dy), EPS)
    t = dy * w
    dw, c = (dy * n).sum(0), (t * n).mean(-1, keepdims=True)
    size = (np.abs(dy) * dn).sum(0) + (rows + 700) * np.abs(dy * n).sum(0)
    assert (np.abs(host(g["dweight"]) - dw) <= U * size + 1e-30).all()
    dx = inv * (t - t.mean(-1, keepdims=True) - n * c)
    at, an = np.abs(t), np.abs(n)
    m = lambda z: z.mean(-1, keepdims=True)  # noqa: E731
    size = inv * (48 * at + 48 * m(at) + 48 * an * m(at * an) + an * (24 * m(at * an) + m(at * dn))
                  + dn * m(at * an)) + np.abs(dx)
    assert (np.abs(host(g["dx"]) - dx) <= U * size + 1e-30).all()
