"""The float64 linear-attention reference against independent forms (CPU):
the quadratic form with masks, central differences of its gradients, splitting
a sequence, and the step."""
import numpy as np
import pytest

from oracle import linattn
from state_space_model_analytic_gb300 import synth


def small(T=7, lens=None, decays=(-0.3, -2.0), B=2, H=4, G=2, K=8, V=8):
    inp = synth.linattn_inputs(B, T, H, G, K, V, "f32", 5, decays)
    return inp


def test_forward_is_the_masked_quadratic_form():
    inp = small(T=9, decays=(-0.3, 0.0))
    o, _ = linattn.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state0"], 0.7)
    q, k = (np.repeat(inp[x], 2, axis=2) for x in "qk")
    i = np.arange(9)
    m = np.where(i[:, None] >= i[None], np.exp(inp["log_decay"][:, None, None] *
                                               np.maximum(i[:, None] - i[None], 0)), 0)
    ref = 0.7 * np.einsum("bihk,bjhk,hij,bjhv->bihv", q, k, m, inp["v"])
    lead = np.exp(inp["log_decay"][None] * (i[:, None] + 1))
    ref += 0.7 * np.einsum("bihk,bhvk,ih->bihv", q, inp["state0"], lead)
    np.testing.assert_allclose(o, ref, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("lens", [None, [3, 0]])
def test_gradients_are_central_differences(lens):
    inp = small(T=4, B=2, H=2, G=1)
    names = {"q": "dq", "k": "dk", "v": "dv", "state0": "dstate0"}

    def loss(x):
        o, S = linattn.forward(x["q"], x["k"], x["v"], x["log_decay"], x["state0"], 0.6, lens)
        return (o * inp["do"]).sum() + (S * inp["dstate"]).sum()

    g = linattn.backward(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state0"], inp["do"],
                         inp["dstate"], 0.6, lens)
    h = 1e-4
    for name, dn in names.items():
        num = np.zeros_like(np.asarray(inp[name], dtype=np.float64))
        for at in np.ndindex(num.shape):
            hi, lo = dict(inp), dict(inp)
            hi[name], lo[name] = np.array(inp[name], float), np.array(inp[name], float)
            hi[name][at] += h
            lo[name][at] -= h
            num[at] = (loss(hi) - loss(lo)) / (2 * h)
        # the loss is linear in every single element: no truncation error, only
        # the rounding of a sum of about 1e3, 2^-52 * 1e3 / 1e-4
        np.testing.assert_allclose(g[dn], num, rtol=0, atol=1e-7)


def test_a_sequence_in_two_parts_and_by_steps():
    inp = small(T=11)
    q, k, v, la = (inp[x] for x in ("q", "k", "v", "log_decay"))
    o, S = linattn.forward(q, k, v, la, inp["state0"])
    o1, S1 = linattn.forward(q[:, :4], k[:, :4], v[:, :4], la, inp["state0"])
    o2, S2 = linattn.forward(q[:, 4:], k[:, 4:], v[:, 4:], la, S1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-12)
    s = inp["state0"]
    for t in range(11):
        y, s = linattn.step(q[:, t], k[:, t], v[:, t], la, s)
        np.testing.assert_allclose(y, o[:, t], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(s, S, rtol=1e-12, atol=1e-12)


def test_no_memory_and_short_rows():
    inp = small(T=5, decays=(-np.inf, -0.1))
    o, S = linattn.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state0"], 1.0, [0, 5])
    assert not o[0].any() and np.array_equal(S[0], inp["state0"][0])
    ref = np.einsum("tgk,tgk->tg", inp["q"][1], inp["k"][1])[:, 0, None] * inp["v"][1][:, 0]
    np.testing.assert_allclose(o[1, :, 0], ref, rtol=1e-12, atol=1e-12)
