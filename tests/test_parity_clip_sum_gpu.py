"""The gradient norm over many equal squares, where roundings that share a
direction would add up.

Tolerance: with u = 2^-24, sums of at most eight squares, each rounded once as it
is added, and two more additions reach a running sum that keeps its own rounding
errors, and fp64 from there: the sum is within 10 u, its root within 5 u, and n is
rounded once.  8 u leaves room for terms of second order."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


@pytest.mark.parametrize("value", [1e-3, 0.7, 1.1])
@pytest.mark.parametrize("kind,count", [("bf16", 4000000007), ("bf16", 300000001), ("f32", 1000000003),
                                        ("f32", 1000003)])
def test_equal_gradients(kind, count, value):
    """Up to 8 GB in one tensor: offsets past 32 bits, and thousands of squares a
    thread."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    g = torch.full((count,), value, dtype=torch.bfloat16 if kind == "bf16" else torch.float32,
                   device="cuda")
    v = float(g[0].double())
    n = float(ssd.clip_grad_norm([g], float("inf")))
    ref = v * count ** 0.5
    assert abs(n - ref) <= 8 * 2.0 ** -24 * ref, (n - ref) / ref * 2.0 ** 24
    assert float(g[-1].double()) == v


def test_a_large_tensor_is_scaled_to_its_end():
    import torch
    import state_space_model_analytic_gb300 as ssd
    count = 2200000011  # more than 2^31 elements
    g = torch.ones(count, dtype=torch.bfloat16, device="cuda")
    ssd.clip_grad_norm([g], 0.5 * count ** 0.5, eps=0.0)
    assert bool((g == 0.5).all())
