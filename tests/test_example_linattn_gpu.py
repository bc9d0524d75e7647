"""The linear-attention example end to end: it learns, its token steps agree
with its prompt pass, and it continues prompts of different lengths."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def test_steps_agree_with_the_prompt_pass():
    """The same tokens as one prompt and as a prompt and steps: logits agree to
    the bf16 roundings of the layers (2^-8 of activations of order one, a dozen
    of them in quadrature)."""
    import torch
    import linattn_lm
    model = linattn_lm.Model()
    gen = torch.Generator("cuda").manual_seed(5)
    tokens = linattn_lm.batch(gen, 6, 50)
    full = torch.full((6,), 50, dtype=torch.int32, device="cuda")
    want, _ = model.read(tokens, full)
    got, states = model.read(tokens[:, :40].contiguous(), torch.full_like(full, 40))
    for t in range(40, 50):
        got = model.step(tokens[:, t], states)
    assert float((got - want).norm() / want.norm()) <= 2.0 ** -5


def test_it_learns_and_continues():
    import linattn_lm
    losses, right = linattn_lm.main(steps=200, quiet=True)
    # chance is ln 32 = 3.47 and the best mixture of the four permutations ln 4 = 1.39;
    # the first of a row's 96 tokens cannot be known (3.47 / 96 = 0.04)
    assert losses[0] > 3.0 and losses[-1] < 0.5, (losses[0], losses[-1])
    assert right > 0.9
