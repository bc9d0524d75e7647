"""The block norms' backward with the forward's statistics, which are those of the
unrounded residual: with a residual stored in bf16 they are not those of what is
stored.  Tolerances as in the tests of every output: 64 roundings of fp32 of the
terms' magnitudes, and as many more as rows are added, and one rounding of the
output."""
import numpy as np
import pytest

from oracle import layer
from test_parity_blocknorm_gpu import _built, check, dev, host, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width", [(17, 256), (300, 2048), (3, 4099), (9, 8192), (1000, 8)])
@pytest.mark.parametrize("gate", [True, False])
def test_a_bf16_residual_s_statistics(rows, width, gate):
    import state_space_model_analytic_gb300 as ssd
    x = inputs(rows, width, "bf16", "bf16", rows * width)
    z = x["z"] if gate else None
    w = dev(x["w_post"]), dev(x["res_scale"]), dev(x["w_pre"])
    y, zz = dev(x["y"], "bf16"), dev(z, "bf16")
    new, _, stats = ssd.block_norm_forward(dev(x["residual"], "bf16"), y, zz, *w, 1e-5)
    exact, em = layer.block_norm_forward(x["residual"], x["y"], z, x["w_post"], x["res_scale"],
                                         x["w_pre"], 1e-5)
    inv = [1.0 / np.sqrt((t ** 2).mean(-1, keepdims=True) + 1e-5) for t in (x["y"], exact["residual"])]
    # of an inverse root of a mean of squares t^2 with terms of magnitude m
    mag = [2 * inv[0], inv[1] * (1 + inv[1] ** 2 * (np.abs(exact["residual"]) * em["residual"])
                                 .mean(-1, keepdims=True))]
    for i in range(2):
        assert (np.abs(host(stats)[:, i:i + 1] - inv[i]) <= 64 * 2.0 ** -24 * mag[i]).all()
    ref, mag = layer.block_norm_backward(host(new), x["y"], z, x["w_post"], x["res_scale"], x["w_pre"],
                                         1e-5, x["dx"], x["dnew"], stats=inv)
    g = ssd.block_norm_backward(new, y, zz, *w, 1e-5, dev(x["dx"], "bf16"), dev(x["dnew"], "bf16"), stats)
    for n in ref:
        assert (g[n] is None) == (ref[n] is None), n
        if ref[n] is not None:
            weights = n in ("dw_post", "dres_scale", "dw_pre")
            check(host(g[n]), ref[n], mag[n], "f32" if weights else "bf16", rows + 64 if weights else 0)
