"""The float64 delta-rule reference against independent forms (CPU): the chunk
form, differences of its gradients, splitting a sequence, and the step."""
import numpy as np
import pytest

from oracle import delta
from state_space_model_analytic_gb300 import synth

NAMES = ("q", "k", "v", "log_decay", "beta")


def small(T=7, B=2, H=4, G=2, K=8, V=8, decays=None):
    return synth.delta_inputs(B, T, H, G, K, V, "f32", 5, decays)


def test_forward_is_the_triangular_system():
    """(I + L beta) E = V - e^g K S^T over the whole row, solved at once."""
    inp = small(T=9)
    o, S, _, _ = delta.forward(*(inp[n] for n in NAMES), inp["state0"], 0.7)
    q, k = (np.repeat(inp[x], 2, axis=2) for x in "qk")
    for b in range(2):
        for h in range(4):
            g = np.cumsum(inp["log_decay"][b, :, h])
            gam = np.exp(g[:, None] - g[None])
            L = np.tril(gam * (k[b, :, h] @ k[b, :, h].T), -1)
            be = inp["beta"][b, :, h]
            S0 = inp["state0"][b, h]
            E = np.linalg.solve(np.eye(9) + L * be, inp["v"][b, :, h] - np.exp(g)[:, None] * (k[b, :, h] @ S0.T))
            P = np.tril(gam * (q[b, :, h] @ k[b, :, h].T))
            ref = 0.7 * (np.exp(g)[:, None] * (q[b, :, h] @ S0.T) + P @ (be[:, None] * E))
            np.testing.assert_allclose(o[b, :, h], ref, rtol=1e-10, atol=1e-12)
            end = np.exp(g[-1]) * S0 + (be[:, None] * E).T @ (np.exp(g[-1] - g)[:, None] * k[b, :, h])
            np.testing.assert_allclose(S[b, h], end, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("lens", [None, [3, 0]])
def test_gradients_are_central_differences(lens):
    inp = small(T=4, H=2, G=1)

    def loss(x):
        o, S, _, _ = delta.forward(*(x[n] for n in NAMES), x["state0"], 0.6, lens)
        return (o * inp["do"]).sum() + (S * inp["dstate"]).sum()

    g, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"], 0.6, lens)
    h = 2.0 ** -13
    for name in NAMES + ("state0",):
        num = np.zeros_like(np.asarray(inp[name], dtype=np.float64))
        for at in np.ndindex(num.shape):
            y = []
            for d in (2 * h, h, -h, -2 * h):
                x = dict(inp)
                x[name] = np.array(inp[name], float)
                x[name][at] += d
                y.append(loss(x))
            num[at] = (8 * (y[1] - y[2]) - (y[0] - y[3])) / (12 * h)
        # fourth order: h^4 = 2^-52 of derivatives of size 1e2; rounding 2^-52 * 1e3 / h
        np.testing.assert_allclose(g["d" + name], num, rtol=0, atol=2e-8)


def test_a_sequence_in_two_parts_and_by_steps():
    inp = small(T=11)
    whole = [inp[n] for n in NAMES]
    o, S, _, _ = delta.forward(*whole, inp["state0"])
    o1, S1, _, _ = delta.forward(*(x[:, :4] for x in whole), inp["state0"])
    o2, S2, _, _ = delta.forward(*(x[:, 4:] for x in whole), S1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-12)
    s = inp["state0"]
    for t in range(11):
        y, s = delta.step(*(x[:, t] for x in whole), s)
        np.testing.assert_allclose(y, o[:, t], rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(s, S, rtol=1e-12, atol=1e-12)


def test_without_writing_and_with_whole_writing():
    """beta = 0 leaves the decayed state; beta = 1 with a unit key stores v exactly."""
    inp = small(T=5)
    zero = np.zeros_like(inp["beta"])
    o, S, _, _ = delta.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"], zero, inp["state0"])
    a = np.exp(inp["log_decay"].sum(1))[..., None, None]
    np.testing.assert_allclose(S, a * inp["state0"], rtol=1e-12, atol=1e-12)
    k = np.repeat(inp["k"][:, -1], 2, axis=1)
    k1 = inp["k"] / np.sqrt((inp["k"] ** 2).sum(-1, keepdims=True))
    _, S, _, _ = delta.forward(inp["q"], k1, inp["v"], inp["log_decay"], zero + 1, inp["state0"])
    k = np.repeat(k1[:, -1], 2, axis=1)
    np.testing.assert_allclose(np.einsum("bhvk,bhk->bhv", S, k), inp["v"][:, -1], rtol=1e-12, atol=1e-12)


def test_no_memory_and_short_rows():
    inp = small(T=5, decays=(-np.inf,))
    o, S, _, _ = delta.forward(*(inp[n] for n in NAMES), inp["state0"], 1.0, [0, 5])
    assert not o[0].any() and np.array_equal(S[0], inp["state0"][0])
    q, k = (np.repeat(inp[x], 2, axis=2)[1] for x in "qk")
    ref = (np.einsum("thk,thk->th", q, k) * inp["beta"][1])[..., None] * inp["v"][1]
    np.testing.assert_allclose(o[1], ref, rtol=1e-12, atol=1e-12)
