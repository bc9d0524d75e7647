"""Linear attention against the float64 reference by root mean squares, head by
head, so that a slowly decaying head is not lost among the others and
cancellation between terms does not widen the bound.

Tolerances, relative to the root mean square of a head's (or a group's) values.

bf16: what a kernel rounds to bf16 is rounded once by at most 2^-8, evenly over
that interval, so by 2^-8 / sqrt(3) = 0.0023 in the mean or less.  An output is the
sum of a part through the scores and one through the state, of which each has one
operand rounded so (a rounded weight in front of another operand of zero mean
gives that much of the sum, in the mean), and is rounded itself: at most sqrt(2)
times 0.0023 = 0.0033.  2^-8 = 0.0039 is allowed.

The fp32 states of bf16 operands: the weighted operand is exact to 2^-24, its
products are added to an accumulator eight times a chunk, each time with an error
of at most 2^-23 of it (the instructions cut off): 2^-20 if all went one way.

fp32: two products after one another whose operands have an error of a few 2^-24,
as in the forward, where 8 x 2^-24 is allowed; a group's sum adds at most a
rounding a head."""
import numpy as np
import pytest

from oracle import linattn
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


def dev(a, dtype="f32"):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def worst(got, ref, axis):
    """The largest relative error of a head, [..., heads, ...] at `axis`."""
    got = np.moveaxis(got.double().cpu().numpy(), axis, 0)
    ref = np.moveaxis(ref, axis, 0)
    n = ref.shape[0]
    err = np.sqrt(((got - ref) ** 2).reshape(n, -1).mean(1))
    return float((err / np.sqrt((ref ** 2).reshape(n, -1).mean(1))).max())


# B, T, H, G, K, V, lens, decays
CASES = [
    (2, 700, 4, 2, 64, 64, None, (-0.01, -0.5, -0.002, -3.0)),
    (2, 1100, 3, 3, 128, 128, None, (-0.004, -0.1, -2.0)),
    (3, 520, 4, 1, 128, 64, (520, 129, 400), (-0.02, -0.3, -0.001, 0.0)),
    (2, 530, 3, 3, 80, 40, None, (-0.03, -0.7, -0.005)),
    (1, 4100, 2, 1, 64, 64, None, (-0.002, -0.05)),  # shared out over segments
]
ids = [f"b{c[0]}t{c[1]}h{c[2]}g{c[3]}k{c[4]}v{c[5]}{'lens' if c[6] else ''}" for c in CASES]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_every_head(case, dtype):
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, lens, decays = case
    inp = synth.linattn_inputs(B, T, H, G, K, V, dtype, 300 + T, decays)
    q, k, v, do = (dev(inp[x], dtype) for x in ("q", "k", "v", "do"))
    la, s0, ds = (dev(inp[x]) for x in ("log_decay", "state0", "dstate"))
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, S = ssd.linattn_forward(q, k, v, la, s0, scale=0.25, lens=ln)
    g = ssd.linattn_backward(q, k, v, la, s0, do, ds, scale=0.25, lens=ln)
    a = (inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state0"])
    ro, rS = linattn.forward(*a, 0.25, lens)
    rg = linattn.backward(*a, inp["do"], inp["dstate"], 0.25, lens)
    out = 2.0 ** -8 if dtype == "bf16" else 8 * U
    state = 2.0 ** -20 if dtype == "bf16" else 8 * U
    assert worst(o, ro, 2) <= out
    assert worst(S, rS, 1) <= state
    assert worst(g["dv"], rg["dv"], 2) <= out
    assert worst(g["dstate0"], rg["dstate0"], 1) <= state
    for n in ("dq", "dk"):
        assert worst(g[n], rg[n], 2) <= out + (H // G) * U, n
