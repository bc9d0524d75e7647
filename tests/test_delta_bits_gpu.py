"""How many bits the gated delta rule's results keep: outputs that are rounded once, keys
that are alike, operands whose elements, steps or columns differ by powers of two.

Tolerances.  A value held in 32 bits enters a product with 22 bits, off by 2^-23 of
itself at most; a sum passes through a few dozen such terms and truncations of 2^-23,
which as signs differ leave a few 2^-22 of its root mean square: 2^-19 is allowed, a
factor of eight.  An element of 10^5 is off by five times that root mean square, and
gradients sum up what two walks leave: 2^-16 for single elements.  A bf16 result is
rounded by 2^-8 of itself besides."""
import numpy as np
import pytest

from oracle import delta
from state_space_model_analytic_gb300 import synth
from test_parity_delta_gpu import NAMES, _built, dev, host, operands  # noqa: F401

pytestmark = pytest.mark.gpu
RMS, ONE = 2.0 ** -19, 2.0 ** -16
GRADS = ("dq", "dk", "dv", "dlog_decay", "dbeta", "dstate0")


def recurrence(inp, state0=None, scale=1.0):
    """o and the final state in 64 bits, step by step."""
    import torch
    t = lambda x: torch.from_numpy(np.asarray(x, dtype=np.float64)).cuda()  # noqa: E731
    q, k, v, la, be = (t(inp[n]) for n in NAMES)
    B, T, H, V = v.shape
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    S = torch.zeros(B, H, V, k.shape[-1], dtype=torch.float64, device="cuda")
    S = S if state0 is None else t(state0)
    o = torch.empty(B, T, H, V, dtype=torch.float64, device="cuda")
    for i in range(T):
        S = S * la[:, i].exp()[..., None, None]
        e = v[:, i] - (S @ k[:, i, :, :, None])[..., 0]
        S = S + (be[:, i, :, None] * e)[..., None] * k[:, i, :, None, :]
        o[:, i] = scale * (S @ q[:, i, :, :, None])[..., 0]
    return o.cpu().numpy(), S.cpu().numpy()


def rms(x, axes=None):
    return np.sqrt(np.mean(x * x, axis=axes, keepdims=axes is not None))


def close(got, ref, axes=None, most=RMS):
    """Root mean square of the errors against that of the values, over `axes`."""
    assert np.isfinite(got).all()
    off = rms(got - ref, axes) / np.maximum(rms(ref, axes), 1e-300)
    assert (off <= most).all(), float(np.log2(off.max()))


def rounded_once(got, ref, axes):
    """Off by the rounding to bf16 and ONE of the root mean square over `axes`."""
    assert np.isfinite(got).all()
    over = np.maximum(np.abs(got - ref) - 2.0 ** -8 * np.abs(ref), 0) / rms(ref, axes)
    assert (over <= ONE).all(), float(np.log2(over.max()))


# heads, groups, K, V: four, two and one warp to 16 rows of a state, o by the walking warps
# and by others
SHAPES = [(3, 3, 64, 64), (50, 50, 64, 64), (80, 80, 64, 64),
          (3, 1, 128, 64), (50, 25, 128, 64), (80, 80, 128, 64), (40, 40, 128, 128), (160, 8, 72, 24)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_outputs_are_rounded_once(shape):
    import state_space_model_analytic_gb300 as ssd
    H, G, K, V = shape
    inp = synth.delta_inputs(1, 200, H, G, K, V, "bf16", 81)
    o, S = ssd.delta_rule_forward(*operands(inp, "bf16"), dev(inp["state0"]))
    ro, rS = recurrence(inp, inp["state0"])
    rounded_once(host(o), ro, (1, 3))
    close(host(S), rS, (2, 3))


@pytest.mark.parametrize("shape", [(3, 3, 64, 64), (4, 2, 128, 128), (2, 2, 72, 40)], ids=str)
def test_gradients_are_rounded_once(shape):
    import state_space_model_analytic_gb300 as ssd
    H, G, K, V = shape
    inp = synth.delta_inputs(1, 200, H, G, K, V, "bf16", 82)
    g = ssd.delta_rule_backward(*operands(inp, "bf16"), dev(inp["state0"]), dev(inp["do"], "bf16"),
                                dev(inp["dstate"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    for n in ("dq", "dk", "dv"):
        rounded_once(host(g[n]), ref[n], (1, 3))


@pytest.mark.parametrize("kind", ["alike", "noisy", "signs"])
@pytest.mark.parametrize("shape", [(80, 128, 64), (3, 128, 64), (80, 64, 64)], ids=str)
def test_states_of_alike_keys(shape, kind):
    """Keys of length 1 that hardly differ, differ by a third, or have elements of the
    same size: the triangular system's inverse and its matrix are of very different size.
    (Where one key's share is written over and over, what is left of it is small: the
    errors go by the largest that the state's row has held, hence by v's size here.)"""
    import state_space_model_analytic_gb300 as ssd
    H, K, V = shape
    inp = synth.delta_inputs(1, 512, H, H, K, V, "bf16", 83)
    rng = np.random.default_rng(84)
    k = {"alike": 1.0 + 0.05 * inp["k"], "noisy": 1.0 + 0.3 * rng.standard_normal(inp["k"].shape),
         "signs": np.sign(rng.standard_normal(inp["k"].shape))}[kind]
    inp["k"] = synth.round_to(k / np.sqrt((k * k).sum(-1, keepdims=True)), "bf16")
    inp["beta"] = np.ones_like(inp["beta"])
    inp["log_decay"] = np.zeros_like(inp["log_decay"])
    o, S = ssd.delta_rule_forward(*operands(inp, "bf16"))
    ro, rS = recurrence(inp)
    close(host(S), rS, (2, 3))
    rounded_once(host(o), ro, (1, 3))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_gradient_stays_in_its_column(dtype, bad):
    """Columns of v are independent of one another on the way back too: dv and dstate0
    are what they are without the bad value in all other columns."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 200, 2, 1, 64, 64, dtype, 85)
    x, do = operands(inp, dtype), dev(inp["do"], dtype)
    s0, ds = dev(inp["state0"]), dev(inp["dstate"])
    g = ssd.delta_rule_backward(*x, s0, do, ds)
    do[0, 70, 1, 5] = bad
    h = ssd.delta_rule_backward(*x, s0, do, ds)
    assert not torch.isfinite(h["dv"][0, :71, 1, 5]).any()
    assert not torch.isfinite(h["dstate0"][0, 1, 5]).any()
    keep = torch.ones_like(g["dv"], dtype=torch.bool)
    keep[0, :, 1, 5] = False
    assert torch.equal(h["dv"][keep], g["dv"][keep])
    keep = torch.ones_like(g["dstate0"], dtype=torch.bool)
    keep[0, 1, 5] = False
    assert torch.equal(h["dstate0"][keep], g["dstate0"][keep])


@pytest.mark.parametrize("H", [2, 80])
def test_columns_of_different_size(H):
    """dout's columns from 1 to 2^-40: each column's dv and dstate0 keep their bits."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 130, H, H, 64, 64, "f32", 86)
    inp["do"] = inp["do"] * np.exp2(-(np.arange(64) % 41.0))
    g = ssd.delta_rule_backward(*operands(inp, "f32"), None, dev(inp["do"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), None, inp["do"])
    close(host(g["dv"]), ref["dv"], (0, 1))
    close(host(g["dstate0"]), ref["dstate0"], (0, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_a_query_do_not_depend_on_it(dtype):
    """dq is the state's product with dout: queries of any size (2^-30 ... 2^30, zero)
    have the same, bit for bit; and dv and dk go by what the steps read."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 150, 3, 3, 64, 128, dtype, 87)
    rng = np.random.default_rng(88)
    q, k, v, la, be = operands(inp, dtype)
    s0, do = dev(inp["state0"]), dev(inp["do"], dtype)
    f = np.exp2(rng.integers(-30, 31, (2, 150, 3, 1)))
    f[:, 7] = 0
    g = ssd.delta_rule_backward(q, k, v, la, be, s0, do)
    h = ssd.delta_rule_backward((q.float() * dev(f)).to(q.dtype), k, v, la, be, s0, do)
    assert torch.equal(g["dq"], h["dq"])
    inp["q"] = inp["q"] * f
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"])
    # (f32 results of the rows before the largest reads; a bf16 one is rounded besides)
    for n in ("dk", "dv"):
        close(host(h[n]), ref[n], (1, 3), 2.0 ** -9 if dtype == "bf16" else RMS)


def test_gradients_of_short_keys():
    """Steps whose keys are 2^-30 of the others': their dk goes by v and the state's
    gradient, not by the key."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 150, 2, 2, 64, 64, "f32", 89)
    inp["k"][:, 3::7] *= 2.0 ** -30
    g = ssd.delta_rule_backward(*operands(inp, "f32"), dev(inp["state0"]), dev(inp["do"]), dev(inp["dstate"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    close(host(g["dk"])[:, 3::7], ref["dk"][:, 3::7])
    for n in GRADS[:3]:
        close(host(g[n]), ref[n])


def spread(n, least):
    """1 ... 2^-least over n elements, in an order that is not theirs."""
    return np.exp2(-(np.arange(n) * 7 % (least + 1.0)))


@pytest.mark.parametrize("H", [2, 80])
def test_elements_of_different_size(H):
    """fp32 rows of k and q whose elements are 1 ... 2^-14 of the largest: each column
    of the state, of dk and of dq keeps its bits."""
    import state_space_model_analytic_gb300 as ssd
    K = 64
    inp = synth.delta_inputs(1, 130, H, H, K, 64, "f32", 90)
    c = spread(K, 14)
    for n in "qk":
        x = inp[n] * c
        inp[n] = synth.round_to(x / np.sqrt((x * x).sum(-1, keepdims=True)), "f32")
    x = operands(inp, "f32")
    o, S = ssd.delta_rule_forward(*x)
    ro, rS = recurrence(inp)
    close(host(o), ro, (1, 3))
    close(host(S), rS, (1, 2))
    if H > 2:
        return
    g = ssd.delta_rule_backward(*x, None, dev(inp["do"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), None, inp["do"])
    for n in ("dq", "dk"):
        close(host(g[n]), ref[n], (0, 1, 2))


def test_columns_against_one_another():
    """Columns of v of 1 ... 2^-12 and of dout of 1 ... 2^12: every column has the same
    share in dq, dk and the gates' gradients."""
    import state_space_model_analytic_gb300 as ssd
    V = 128
    inp = synth.delta_inputs(1, 130, 2, 2, 64, V, "f32", 91)
    c = spread(V, 12)
    plain = {n: np.array(inp[n]) for n in inp}
    inp["v"], inp["do"] = inp["v"] * c, inp["do"] / c
    g = ssd.delta_rule_backward(*operands(inp, "f32"), None, dev(inp["do"]))
    ref, _ = delta.backward(*(plain[n] for n in NAMES), None, plain["do"])
    for n in ("dq", "dk", "dbeta"):
        close(host(g[n]), ref[n])


def test_steps_of_different_size():
    """fp32 douts of 1 ... 2^-14 by step (weighted losses): dv of every step keeps its
    bits."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 130, 2, 2, 64, 64, "f32", 92, (-0.5, -0.1))
    inp["do"] = inp["do"] * np.exp2(-np.arange(130) * 14.0 / 130)[:, None, None]
    g = ssd.delta_rule_backward(*operands(inp, "f32"), None, dev(inp["do"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), None, inp["do"])
    close(host(g["dv"]), ref["dv"], (2, 3), 2.0 ** -17)  # (of 128 elements each)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_zeros_before_small_ones(dtype):
    """v, the state and dout zero in the first 64 columns, 2^-70 in the others."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 100, 2, 2, 64, 128, dtype, 93)
    for n in ("v", "do", "state0", "dstate"):
        x = np.array(inp[n])
        if n in ("v", "do"):
            x[..., :64] = 0
        else:
            x[..., :64, :] = 0
        inp[n] = x
    f = 2.0 ** -70
    x = operands(inp, dtype)
    a = ssd.delta_rule_backward(*x, dev(inp["state0"]), dev(inp["do"], dtype), dev(inp["dstate"]))
    x[2] = x[2] * f
    b = ssd.delta_rule_backward(*x, dev(inp["state0"] * f), dev(inp["do"] * f, dtype),
                                dev(inp["dstate"] * f))
    # dq, dk and the gates' are products of two such factors, 2^-140: zero, or of a few bits
    tiny = 2.0 ** -139
    for n in ("dq", "dk", "dlog_decay", "dbeta"):
        got, most = host(b[n]), np.abs(host(a[n])).max() * tiny
        assert np.isfinite(got).all() and np.abs(got).max() <= most, n
    for n in ("dv", "dstate0"):
        assert np.array_equal(host(a[n]) * f, host(b[n])), n


# as SHAPES, and groups and two pieces of v for the gradients
PATHS = [(3, 3, 64, 64), (50, 25, 128, 64), (80, 80, 128, 64), (80, 40, 64, 64), (4, 2, 128, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PATHS, ids=str)
def test_sums_keep_their_bits_on_every_path(shape, dtype):
    """Outputs and gradients by their root mean squares, head by head.  (The terms of
    dlog_decay cancel to a thirtieth and less of their size: 2^-17.  A bf16 result
    between 1 and 2 is rounded by up to 2^-8, 2^-8 / sqrt(3) in the root mean square, and
    is 1.5 itself: below 2^-9.)"""
    import state_space_model_analytic_gb300 as ssd
    H, G, K, V = shape
    inp = synth.delta_inputs(1, 130, H, G, K, V, dtype, 94)
    x, s0 = operands(inp, dtype), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0)
    g = ssd.delta_rule_backward(*x, s0, dev(inp["do"], dtype), dev(inp["dstate"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    ro, rS = recurrence(inp, inp["state0"])
    over = {"state": (2, 3), "dstate0": (2, 3), "dlog_decay": 1, "dbeta": 1}
    for n, got, want in (("o", o, ro), ("state", S, rS), *((n, g[n], ref[n]) for n in GRADS)):
        most = 2.0 ** -9 if dtype == "bf16" and n in ("o", "dq", "dk", "dv") else RMS
        close(host(got), want, over.get(n, (1, 3)), 2.0 ** -17 if n == "dlog_decay" else most)


@pytest.mark.parametrize("scale", [-3.7, 0.0, 2.0 ** -40, 1e9])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(dtype, scale):
    """Any scale of o: gradients against the reference; with 0 those of the state alone."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 100, 4, 2, 64, 128, dtype, 95)
    g = ssd.delta_rule_backward(*operands(inp, dtype), dev(inp["state0"]), dev(inp["do"], dtype),
                                dev(inp["dstate"]), scale=scale)
    scale = float(np.float32(scale))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"], scale)
    if scale == 0:
        assert not host(g["dq"]).any()
    for n in GRADS[scale == 0:]:
        most = 2.0 ** -9 if dtype == "bf16" and n in ("dq", "dk", "dv") else RMS
        close(host(g[n]), ref[n], None, 2.0 ** -17 if n == "dlog_decay" else most)


@pytest.mark.parametrize("f", [2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_queries(dtype, f):
    """q times f and dout divided by it: o and dq change by that factor, nothing else
    does, bit for bit."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 150, 4, 2, 64, 128, dtype, 96)
    q, k, v, la, be = operands(inp, dtype)
    s0, do, ds = dev(inp["state0"]), dev(inp["do"], dtype), dev(inp["dstate"])
    # (a dout that is all bits at 2^-100 too: elements below 2^-20 are left out)
    do = torch.where(do.abs() < 2.0 ** -20, torch.zeros_like(do), do)
    o, S = ssd.delta_rule_forward(q, k, v, la, be, s0)
    o2, S2 = ssd.delta_rule_forward(q * f, k, v, la, be, s0)
    assert torch.equal(o * f, o2) and torch.equal(S, S2)
    g = ssd.delta_rule_backward(q, k, v, la, be, s0, do, ds)
    h = ssd.delta_rule_backward(q * f, k, v, la, be, s0, do * (1 / f), ds)
    assert torch.equal(g["dq"] * (1 / f), h["dq"])
    for n in GRADS[1:]:
        assert torch.equal(g[n], h[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["beta", "v", "do", "q", "k", "all"])
def test_zeros(dtype, what):
    """Write strengths, values, gradients, queries, keys or all of them zero."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 100, 4, 2, 64, 128, dtype, 97)
    for n in ("beta", "v", "do", "q", "k", "state0", "dstate") if what == "all" else (what,):
        inp[n] = np.zeros_like(inp[n])
    x, s0 = operands(inp, dtype), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0)
    g = ssd.delta_rule_backward(*x, s0, dev(inp["do"], dtype), dev(inp["dstate"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    ro, rS = recurrence(inp, inp["state0"])
    for n, got, want in (("o", o, ro), ("state", S, rS), *((n, g[n], ref[n]) for n in GRADS)):
        most = 2.0 ** -9 if dtype == "bf16" and n in ("o", "dq", "dk", "dv") else RMS
        if want.any():
            close(host(got), want, None, 2.0 ** -17 if n == "dlog_decay" else most)
        else:
            assert not host(got).any(), n
