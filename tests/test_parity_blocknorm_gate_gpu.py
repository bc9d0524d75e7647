"""The gate of the block norms over its whole range, element by element.

Rows of ones are their own norm (eps = 0) and weights of one leave silu(z) alone
in r' and its derivative in dz.  Tolerances in units of u = 2^-24 of the value: the
exponential is within 2 ulp (4 u), the sum, the quotient and the products are a
rounding each, the row's norm a few: 16 u.  silu'(z) = s (1 + z (1 - s)) adds the
rounding of 1 - s, at most u / 2 of s, times z, which counts up to z = 17 where
1 - s is below u: 8.5 u more, of the terms' magnitudes: 32 u."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


@pytest.mark.parametrize("width", [1024, 1001, 8192])
def test_fp32_gate_and_its_derivative(width):
    import torch
    import state_space_model_analytic_gb300 as ssd
    z = torch.linspace(-80, 80, 4 * width, device="cuda").view(4, width)
    one, w = torch.ones_like(z), torch.ones(width, device="cuda")
    new, _, _ = ssd.block_norm_forward(torch.zeros_like(z), one, z, w, None, w, 0.0)
    x = z.double().cpu().numpy()
    s = 1.0 / (1.0 + np.exp(-x))
    err = np.abs(new.double().cpu().numpy() - x * s) / np.abs(x * s)
    assert err.max() <= 16 * U, err.max() / U
    g = ssd.block_norm_backward(one, one, z, w, None, w, 0.0, torch.zeros_like(z), one)
    d, mag = s * (1 + x * (1 - s)), s * (1 + np.abs(x) * (1 - s))
    err = np.abs(g["dz"].double().cpu().numpy() - d) / mag
    assert err.max() <= 32 * U, err.max() / U
