"""GPU parity of layer norm against its definition in float64.

Tolerances.  With n = (x - mean) / sqrt(var + eps), the mean is a sum of `width`
fp32 terms in a tree of at most 8 + 10 additions: off by 20 * 2^-24 of mean |x|; so is
the variance of its terms.  y = n w + b is off by
  2^-24 (40 |n w| + 24 mean|x| inv |w| + 2 |b|)
and a bf16 output by 2^-8 of itself more.  Gradients see the same errors in n and two
more such means; sums over the rows add 2^-24 a term of the sum of magnitudes, at most
rows / 8 + 600 + 8 of them in a chain, here bounded by (rows + 700) 2^-24."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def dev(a, dtype="f32"):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.double().cpu().numpy()


def inputs(rows, width, dtype, seed, offset=0.7):
    from state_space_model_analytic_gb300 import synth
    rng = np.random.default_rng(seed)
    r = lambda a: synth.round_to(a, dtype)  # noqa: E731
    f = lambda a: synth.round_to(a, "f32")  # noqa: E731
    return {"x": r(rng.standard_normal((rows, width)) * rng.uniform(0.2, 3, width) + offset),
            "w": f(1 + 0.2 * rng.standard_normal(width)), "b": f(0.3 * rng.standard_normal(width)),
            "dy": r(rng.standard_normal((rows, width)))}


def stats(x, eps):
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    return mean, 1.0 / np.sqrt(var + eps)


def reference(i, eps, w, b):
    """values, sizes of their errors in units of 2^-24"""
    x, dy = i["x"], i["dy"]
    w = np.ones(x.shape[-1]) if w is None else w
    mean, inv = stats(x, eps)
    n = (x - mean) * inv
    dn = 40 * np.abs(n) + 24 * np.abs(x).mean(-1, keepdims=True) * inv  # of n
    t = dy * w
    a, c = t.mean(-1, keepdims=True), (t * n).mean(-1, keepdims=True)
    ma, mc = np.abs(t).mean(-1, keepdims=True), np.abs(t * n).mean(-1, keepdims=True)
    dc = 24 * mc + (np.abs(t) * dn).mean(-1, keepdims=True)
    rows = x.shape[0]
    out = {"y": n * w + (0 if b is None else b), "dx": inv * (t - a - n * c),
           "dweight": (dy * n).sum(0), "dbias": dy.sum(0)}
    size = {"y": dn * np.abs(w) + 2 * (0 if b is None else np.abs(b)),
            "dx": inv * (48 * np.abs(t) + 48 * ma + 48 * np.abs(n) * mc + np.abs(n) * dc + dn * mc),
            "dweight": (np.abs(dy) * dn).sum(0) + (rows + 700) * np.abs(dy * n).sum(0),
            "dbias": (rows + 700) * np.abs(dy).sum(0)}
    return out, size


def check(got, ref, size, rounded):
    assert np.isfinite(got).all()
    err, most = np.abs(got - ref), U * size + rounded * np.abs(ref) + 1e-30
    assert not (err > most).any(), float((err / most).max())


CASES = [(1, 1, "f32"), (3, 7, "bf16"), (5, 64, "bf16"), (300, 257, "f32"), (64, 512, "bf16"),
         (17, 1000, "bf16"), (250, 1537, "f32"), (1300, 2048, "bf16"), (9, 4096, "f32"),
         (40, 5001, "bf16"), (33, 8192, "bf16"), (700, 8191, "f32"), (2, 8192, "f32"), (5000, 96, "bf16")]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("rows,width,dtype", CASES)
def test_forward_and_backward(rows, width, dtype, affine):
    import state_space_model_analytic_gb300 as ssd
    i = inputs(rows, width, dtype, rows + width)
    w, b = (i["w"], i["b"]) if affine else (None, None)
    tw, tb = (dev(w), dev(b)) if affine else (None, None)
    x, dy = dev(i["x"], dtype), dev(i["dy"], dtype)
    ref, size = reference(i, EPS, w, b)
    r = 2.0 ** -8 if dtype == "bf16" else U
    y, st = ssd.layer_norm_forward(x, tw, tb, EPS)
    check(host(y), ref["y"], size["y"], r)
    y2, none = ssd.layer_norm_forward(x, tw, tb, EPS, want_stats=False)
    assert none is None and bool((y == y2).all())
    for s in (st, None):
        g = ssd.layer_norm_backward(x, tw, dy, EPS, s)
        check(host(g["dx"]), ref["dx"], size["dx"], r)
        check(host(g["dweight"]), ref["dweight"], size["dweight"], 0)
        check(host(g["dbias"]), ref["dbias"], size["dbias"], 0)


def test_a_large_mean_costs_no_digits():
    """x = 4096 + noise: the variance comes from differences to the mean."""
    import state_space_model_analytic_gb300 as ssd
    i = inputs(64, 2048, "f32", 1, 4096.0)
    ref, size = reference(i, EPS, i["w"], i["b"])
    y, _ = ssd.layer_norm_forward(dev(i["x"]), dev(i["w"]), dev(i["b"]), EPS)
    check(host(y), ref["y"], size["y"], U)


def test_constant_rows_and_a_zero_eps():
    """A constant row is off its mean by rounding at most: n is 0 for values that sum
    exactly, and with eps = 0 NaN, in that row alone."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    x = torch.full((9, 256), 3.0, device="cuda")
    x[4] = torch.randn(256, device="cuda")
    b = torch.randn(256, device="cuda")
    y, _ = ssd.layer_norm_forward(x, None, b, EPS)
    assert torch.equal(y[0], b) and torch.isfinite(y).all()
    y, _ = ssd.layer_norm_forward(x, None, b, 0.0)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[4]).all()
    # rows that fill up a group of rows do not enter the sums
    g = ssd.layer_norm_backward(x[4:5], None, torch.ones_like(x[4:5]), 0.0)
    assert all(torch.isfinite(t).all() for t in g.values())


def test_strided_unaligned_and_in_place():
    import torch
    import state_space_model_analytic_gb300 as ssd
    i = inputs(50, 512, "bf16", 2)
    x, w, b, dy = dev(i["x"], "bf16"), dev(i["w"]), dev(i["b"]), dev(i["dy"], "bf16")
    y, st = ssd.layer_norm_forward(x, w, b, EPS)
    g = ssd.layer_norm_backward(x, w, dy, EPS, st)
    wide = torch.zeros(50, 1024 + 8, dtype=torch.bfloat16, device="cuda")
    ref, size = reference(i, EPS, i["w"], i["b"])
    for at in (0, 8, 3):
        v = wide[:, at:at + 512]
        v.copy_(x)
        z, _ = ssd.layer_norm_forward(v, w, b, EPS)
        check(host(z), ref["y"], size["y"], 2.0 ** -8)
        h = ssd.layer_norm_backward(v, w, dy, EPS, st)
        check(host(h["dx"]), ref["dx"], size["dx"], 2.0 ** -8)
    z = x.clone()
    out, _ = ssd.layer_norm_forward(z, w, b, EPS, out=z)
    assert out is z and torch.equal(z, y)
    for name in ("x", "dy"):
        c = {"x": x.clone(), "dy": dy.clone()}
        h = ssd.layer_norm_backward(c["x"], w, c["dy"], EPS, st, out={"dx": c[name]})
        assert h["dx"] is c[name] and all(torch.equal(h[n], g[n]) for n in g)
    x3 = x.view(5, 10, 512)
    y3, st3 = ssd.layer_norm_forward(x3, w, b, EPS)
    assert st3.shape == (5, 10, 2) and torch.equal(y3.view(50, 512), y)
    h = ssd.layer_norm_backward(x, w, dy, EPS, st, want_dweight=False)
    assert h["dweight"] is None and torch.equal(h["dbias"], g["dbias"])
    h = ssd.layer_norm_backward(x, w, dy, EPS, st, want_dweight=False, want_dbias=False)
    assert torch.equal(h["dx"], g["dx"])


def test_a_bad_row_stays_alone_and_runs_are_equal():
    import torch
    import state_space_model_analytic_gb300 as ssd
    i = inputs(400, 640, "bf16", 3)
    x, w, dy = dev(i["x"], "bf16"), dev(i["w"]), dev(i["dy"], "bf16")
    y, st = ssd.layer_norm_forward(x, w, None, EPS)
    g = ssd.layer_norm_backward(x, w, dy, EPS, st)
    side = torch.cuda.Stream()
    h = ssd.layer_norm_backward(x, w, dy, EPS, st, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g[n], h[n]) for n in g)
    bad = x.clone()
    bad[7, 5] = float("nan")
    z, _ = ssd.layer_norm_forward(bad, w, None, EPS)
    assert torch.isnan(z[7]).all()
    keep = torch.arange(400, device="cuda") != 7
    assert torch.equal(z[keep], y[keep])


def test_refusals():
    import torch
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x, w = z(4, 64), z(64)
    f, b = ssd.layer_norm_forward, ssd.layer_norm_backward
    f(x, w, w, EPS)
    with pytest.raises(nat.SsdError):
        f(z(2, 8193), None, None, EPS)
    with pytest.raises(nat.SsdError):
        f(z(0, 64), w, w, EPS)
    with pytest.raises(nat.SsdError):
        f(x, w, w, -1.0)
    with pytest.raises(nat.SsdError):
        f(x, w, w, float("nan"))
    with pytest.raises(ValueError):
        f(torch.zeros((), device="cuda"), None, None, EPS)
    with pytest.raises(ValueError):
        f(x, z(32), w, EPS)
    with pytest.raises(TypeError):
        f(x, w.bfloat16(), w, EPS)
    with pytest.raises(TypeError):
        f(x.half(), w, w, EPS)
    with pytest.raises(ValueError):
        f(x.t(), None, None, EPS)
    with pytest.raises(ValueError):
        f(x.cpu(), None, None, EPS)
    with pytest.raises(TypeError):
        b(x, w, x.bfloat16(), EPS)
    with pytest.raises(ValueError):
        b(x, w, x, EPS, z(4, 3))
    with pytest.raises(nat.SsdError):
        b(x, w, x, EPS, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
