"""GPU parity of the norms around a block (forward, gradients) against the
float64 reference.

Tolerances: with M the sum of the terms' magnitudes, every output is within 64
roundings of fp32 of its definition (a row's sums are at most 8 + 5 + 32
additions deep, the rest are a dozen products), the weights' gradients within
as many more as rows are added one after another; bf16 outputs are rounded
once more (bf16 has 8 significant bits: at most 2^-8)."""
import numpy as np
import pytest

from oracle import layer
from state_space_model_analytic_gb300 import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def inputs(rows, width, dtype, res, seed):
    rng = np.random.default_rng(seed)
    n = lambda dt, std=1.0: synth.round_to(std * rng.standard_normal((rows, width)), dt)  # noqa: E731
    w = lambda: synth.round_to(rng.uniform(0.5, 1.5, width), "f32")  # noqa: E731
    return {"residual": n(res, 2.0), "y": n(dtype), "z": n(dtype, 3.0), "dx": n(dtype),
            "dnew": n(res), "w_post": w(), "res_scale": w() - 1.0, "w_pre": w()}


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.double().cpu().numpy()


def check(got, ref, mag, dtype, extra=0):
    assert np.isfinite(got).all()
    bound = (64 + extra) * U * mag + (2.0 ** -8 * 1.01 * np.abs(ref) if dtype == "bf16" else 0)
    bad = np.abs(got - ref) > bound + 1e-37
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / (mag + 1e-30)).max()))


CASES = [(1, 1, "f32", "f32"), (3, 7, "bf16", "bf16"), (5, 64, "bf16", "f32"), (9, 65, "f32", "f32"),
         (17, 256, "bf16", "bf16"), (33, 320, "bf16", "f32"), (4, 1000, "f32", "f32"),
         (700, 1001, "bf16", "f32"), (2, 2048, "bf16", "f32"), (1300, 2048, "bf16", "bf16"),
         (6, 4096, "f32", "f32"), (3, 4099, "bf16", "bf16"), (5, 8192, "bf16", "f32"),
         (2, 8191, "f32", "f32"), (3, 8192, "f32", "f32"), (1000, 8, "bf16", "bf16")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}{c[2]}{c[3]}")
@pytest.mark.parametrize("gate,scale", [(True, True), (False, False), (True, False)])
def test_every_output(case, gate, scale):
    import state_space_model_analytic_gb300 as ssd
    rows, width, dtype, res = case
    x = inputs(rows, width, dtype, res, rows + width)
    z = x["z"] if gate else None
    al = x["res_scale"] if scale else None
    w = dev(x["w_post"]), dev(al), dev(x["w_pre"])
    y, zz = dev(x["y"], dtype), dev(z, dtype)
    new, xo, stats = ssd.block_norm_forward(dev(x["residual"], res), y, zz, *w, 1e-5)
    ref, mag = layer.block_norm_forward(x["residual"], x["y"], z, x["w_post"], al, x["w_pre"], 1e-5)
    check(host(new), ref["residual"], mag["residual"], res)
    check(host(xo), ref["x"], mag["x"], dtype)
    stored = host(new)
    dnew = x["dnew"] if scale else None
    ref, mag = layer.block_norm_backward(stored, x["y"], z, x["w_post"], al, x["w_pre"], 1e-5,
                                         x["dx"], dnew)
    g = ssd.block_norm_backward(new, y, zz, *w, 1e-5, dev(x["dx"], dtype), dev(dnew, res))
    for n in ref:
        assert (g[n] is None) == (ref[n] is None), n
        if ref[n] is None:
            continue
        weights = n in ("dw_post", "dres_scale", "dw_pre")
        check(host(g[n]), ref[n], mag[n],
              "f32" if weights else res if n == "dresidual" else dtype, rows + 64 if weights else 0)
    if res == "f32":  # the forward's statistics are those of the stored residual
        g2 = ssd.block_norm_backward(new, y, zz, *w, 1e-5, dev(x["dx"], dtype), dev(dnew, res), stats)
        for n in ref:
            if ref[n] is not None:
                weights = n in ("dw_post", "dres_scale", "dw_pre")
                check(host(g2[n]), ref[n], mag[n],
                      "f32" if weights else res if n == "dresidual" else dtype,
                      rows + 64 if weights else 0)


def test_strided_rows_and_unaligned_tensors():
    """A gate and an output that are slices of a wider projection, and tensors
    that start off a 16-byte boundary, give the same values."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    x = inputs(6, 96, "bf16", "f32", 1)
    w = dev(x["w_post"]), dev(x["res_scale"]), dev(x["w_pre"])
    y, z, r = dev(x["y"], "bf16"), dev(x["z"], "bf16"), dev(x["residual"])
    dx, dn = dev(x["dx"], "bf16"), dev(x["dnew"])
    wide = torch.cat([y, z, y[:, :8]], dim=1)
    a = ssd.block_norm_forward(r, y, z, *w, 1e-5)
    b = ssd.block_norm_forward(r, wide[:, :96], wide[:, 96:192], *w, 1e-5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ga = ssd.block_norm_backward(a[0], y, z, *w, 1e-5, dx, dn)
    gb = ssd.block_norm_backward(a[0], wide[:, :96], wide[:, 96:192], *w, 1e-5, dx, dn)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)

    def off(t):  # the same values one element past a boundary
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    ref, mag = layer.block_norm_forward(x["residual"], x["y"], x["z"], x["w_post"], x["res_scale"],
                                        x["w_pre"], 1e-5)
    c = ssd.block_norm_forward(off(r), off(y), off(z), *(off(t) for t in w), 1e-5)
    check(host(c[0]), ref["residual"], mag["residual"], "f32")
    check(host(c[1]), ref["x"], mag["x"], "bf16")


def test_in_place_residual_and_equal_runs():
    import torch
    import state_space_model_analytic_gb300 as ssd
    x = inputs(2000, 512, "bf16", "bf16", 2)
    w = dev(x["w_post"]), dev(x["res_scale"]), dev(x["w_pre"])
    y, z, r = dev(x["y"], "bf16"), dev(x["z"], "bf16"), dev(x["residual"], "bf16")
    new, xo, _ = ssd.block_norm_forward(r, y, z, *w, 1e-5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2, xo2, _ = ssd.block_norm_forward(r, y, z, *w, 1e-5, out={"residual": r}, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert r2 is r and torch.equal(r, new) and torch.equal(xo, xo2)
    dx, dn = dev(x["dx"], "bf16"), dev(x["dnew"], "bf16")
    g1 = ssd.block_norm_backward(new, y, z, *w, 1e-5, dx, dn)
    g2 = ssd.block_norm_backward(new, y, z, *w, 1e-5, dx, dn)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_rows_of_zeros_and_large_gates():
    import torch
    import state_space_model_analytic_gb300 as ssd
    x = inputs(4, 64, "f32", "f32", 3)
    x["y"][0] = 0.0
    x["residual"][0] = 0.0
    x["z"][1] = 100.0
    x["z"][2] = -100.0
    w = dev(x["w_post"]), dev(x["res_scale"]), dev(x["w_pre"])
    new, xo, _ = ssd.block_norm_forward(dev(x["residual"]), dev(x["y"]), dev(x["z"]), *w, 1e-5)
    ref, mag = layer.block_norm_forward(x["residual"], x["y"], x["z"], x["w_post"], x["res_scale"],
                                        x["w_pre"], 1e-5)
    check(host(new), ref["residual"], mag["residual"], "f32")
    check(host(xo), ref["x"], mag["x"], "f32")
    g = ssd.block_norm_backward(new, dev(x["y"]), dev(x["z"]), *w, 1e-5, dev(x["dx"]))
    assert all(torch.isfinite(t).all() for t in g.values())


def test_refusals():
    import torch
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    y, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    f = ssd.block_norm_forward
    f(y, y, None, w, None, w, 1e-5)
    with pytest.raises(nat.SsdError):
        big = torch.zeros(2, 8193, device="cuda")
        f(big, big, None, big[0], None, big[0], 1e-5)
    with pytest.raises(nat.SsdError):
        f(y, y, None, w, None, w, -1.0)
    with pytest.raises(nat.SsdError):
        f(y[:0], y[:0], None, w, None, w, 1e-5)
    with pytest.raises(TypeError):
        f(y.bfloat16(), y, None, w, None, w, 1e-5)
    with pytest.raises(TypeError):
        f(y.half(), y.half(), None, w, None, w, 1e-5)
    with pytest.raises(TypeError):
        f(y, y, None, w.double(), None, w, 1e-5)
    with pytest.raises(ValueError):
        f(y, y[:2], None, w, None, w, 1e-5)
    with pytest.raises(ValueError):
        f(y, y, y[:, :32], w, None, w, 1e-5)
    with pytest.raises(ValueError):
        f(y, torch.zeros(64, 4, device="cuda").t(), None, w, None, w, 1e-5)
    with pytest.raises(ValueError):
        f(y.cpu(), y.cpu(), None, w, None, w, 1e-5)
    with pytest.raises(nat.SsdError):
        ssd.block_norm_backward(y, y, None, w, None, w, 1e-5, y,
                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
