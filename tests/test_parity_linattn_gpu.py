"""GPU parity of linear attention with a decay for each head (forward,
gradients, single token) against the float64 reference.

Tolerances.  Every output is a sum of products; M is the same sum over
magnitudes (the reference on |inputs|), an upper bound of the sum of the
terms' magnitudes.  In fp32 storage an output accumulates n <= K + V + T
rounded terms with rounded decays (a few 2^-24 each): |error| <=
(n + 64) 2^-24 M.  In bf16 storage the chunk's
scores are rounded once to bf16 for the second product and the output once,
each by at most 2^-8 (8 significant bits) of terms that are together well
below M, and the state operand is carried in two bf16 parts or more (2^-16):
|error| <= 1.1 * 2^-8 M is allowed for all of it; the states, which are fp32
outputs, see only the last: 2^-16 M."""
import numpy as np
import pytest

from oracle import linattn
from state_space_model_analytic_gb300 import synth

pytestmark = pytest.mark.gpu


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


def poison(x, lens):
    """NaN where no step is: an operand's memory past a row's length."""
    if lens is None:
        return x
    x = np.array(x)
    for b, n in enumerate(lens):
        x[b, n:] = np.nan
    return x


def tol(dtype, n, state=False):
    if dtype == "f32":
        return (n + 64) * 2.0 ** -24
    return 2.0 ** -16 if state else 1.1 * 2.0 ** -8


def check(got, ref, mag, t):
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    bad = err > t * mag + 1e-30
    assert not bad.any(), (int(bad.sum()), float((err / np.maximum(mag, 1e-30)).max()), t)


# B, T, H, G, K, V, dtype, lens, decays
CASES = [
    (1, 1, 1, 1, 8, 8, "f32", None, None),
    (2, 3, 2, 1, 16, 8, "bf16", None, None),
    (2, 31, 4, 2, 16, 24, "f32", None, (-0.5, 0.0)),
    (1, 128, 2, 2, 64, 64, "bf16", None, None),
    (2, 129, 3, 3, 64, 64, "bf16", None, (-0.02, -3.0, -40.0)),
    (1, 257, 4, 1, 128, 64, "bf16", None, None),
    (2, 300, 2, 2, 64, 128, "bf16", None, None),
    (1, 391, 2, 1, 128, 128, "bf16", None, (-0.01, -0.2)),
    (2, 200, 2, 2, 80, 40, "bf16", None, None),
    (2, 77, 2, 2, 128, 128, "f32", None, None),
    (1, 640, 2, 2, 64, 64, "f32", None, (-0.003, -1.0)),
    (5, 260, 2, 1, 64, 64, "bf16", (0, 1, 128, 259, 260), None),
    (4, 150, 4, 2, 128, 64, "bf16", (150, 129, 0, 2), (0.0, -0.1, -np.inf, -1e30)),
    (3, 70, 2, 2, 32, 16, "f32", (70, 0, 33), (-np.inf, -0.2)),
    # more (row, chunk, group) units than SMs, whole and ending anywhere
    (8, 1300, 4, 2, 64, 64, "bf16", (0, 1, 128, 129, 640, 1000, 1299, 1300), (-0.01, -0.5)),
    (6, 1100, 3, 3, 128, 128, "bf16", None, (-0.004, -0.1, -2.0)),
    # enough steps for a row to be shared out
    (1, 4100, 1, 1, 64, 64, "bf16", None, (-0.002,)),
    (1, 3000, 2, 1, 128, 128, "bf16", (2999,), (-0.001, -0.3)),
    # fp32: columns of v and rows k that end inside a warp's share, shared out rows
    (3, 190, 4, 2, 80, 40, "f32", (190, 65, 129), (-0.01, -0.4, -5.0, 0.0)),
    (2, 2100, 2, 1, 128, 96, "f32", (2100, 1999), (-0.003, -0.05)),
    (1, 1500, 1, 1, 24, 72, "f32", None, (-0.002,)),
]
ids = [f"b{c[0]}t{c[1]}h{c[2]}g{c[3]}k{c[4]}v{c[5]}{c[6]}{'lens' if c[7] else ''}" for c in CASES]


def inputs(case):
    B, T, H, G, K, V, dtype, lens, decays = case
    return synth.linattn_inputs(B, T, H, G, K, V, dtype, 100 + T, decays)


def magnitudes(inp):
    return {k: v if k == "log_decay" else np.abs(v) for k, v in inp.items()}


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case, with_state):
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, dtype, lens, _ = case
    inp = inputs(case)
    s0 = inp["state0"] if with_state else None
    q, k, v = (dev(poison(inp[x], lens), dtype) for x in "qkv")
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, S = ssd.linattn_forward(q, k, v, dev(inp["log_decay"]), None if s0 is None else dev(s0),
                               scale=0.25, lens=ln)
    ro, rS = linattn.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"], s0, 0.25, lens)
    m = magnitudes(inp)
    mo, mS = linattn.forward(m["q"], m["k"], m["v"], m["log_decay"],
                             None if s0 is None else m["state0"], 0.25, lens)
    check(host(o), ro, mo, tol(dtype, K + V + T))
    check(host(S), rS, mS, tol(dtype, T, True))


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case, with_state):
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, dtype, lens, _ = case
    inp = inputs(case)
    s0, ds = (inp["state0"], inp["dstate"]) if with_state else (None, None)
    q, k, v, do = (dev(poison(inp[x], lens), dtype) for x in ("q", "k", "v", "do"))
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = ssd.linattn_backward(q, k, v, dev(inp["log_decay"]), None if s0 is None else dev(s0), do,
                             None if ds is None else dev(ds), scale=0.25, lens=ln)
    ref = linattn.backward(inp["q"], inp["k"], inp["v"], inp["log_decay"], s0, inp["do"], ds, 0.25,
                           lens)
    m = magnitudes(inp)
    mag = linattn.backward(m["q"], m["k"], m["v"], m["log_decay"], None if s0 is None else m["state0"],
                           m["do"], None if ds is None else m["dstate"], 0.25, lens)
    for name in ("dq", "dk", "dv"):
        check(host(g[name]), ref[name], mag[name], tol(dtype, K + V + T + H))
    check(host(g["dstate0"]), ref["dstate0"], mag["dstate0"], tol(dtype, T, True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_is_the_forward_s_difference(dtype):
    """Along a direction u of all inputs, the fp32 forward's difference quotient
    against the sum of gradients times u.  The loss is a polynomial of degree 4
    in the step; with steps of 2^-6 the central difference's h^2 term is below
    2^-12 of the loss's own scale, taken as the sum of the terms' magnitudes."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(1, 150, 2, 1, 64, 64, "f32", 9, (-0.05, -0.4))
    u = synth.linattn_inputs(1, 150, 2, 1, 64, 64, "f32", 10, (-0.05, -0.4))
    names = {"q": "dq", "k": "dk", "v": "dv", "state0": "dstate0"}
    la = dev(inp["log_decay"])

    def loss(h):
        x = {n: dev(inp[n] + h * u[n]) for n in names}
        o, S = ssd.linattn_forward(x["q"], x["k"], x["v"], la, x["state0"], scale=0.125)
        return float((host(o) * inp["do"]).sum() + (host(S) * inp["dstate"]).sum())

    h = 2.0 ** -6
    num = (loss(h) - loss(-h)) / (2 * h)
    x = {n: dev(inp[n], dtype) for n in ("q", "k", "v", "do")}
    g = ssd.linattn_backward(x["q"], x["k"], x["v"], la, dev(inp["state0"]), x["do"],
                             dev(inp["dstate"]), scale=0.125)
    terms = [(host(g[d]) * u[n]) for n, d in names.items()]
    scale = np.sqrt(sum((t ** 2).sum() for t in terms))
    # bf16: the inputs' and outputs' own roundings, 2^-9 each of four factors, in quadrature
    assert abs(sum(t.sum() for t in terms) - num) <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -8) * scale


def test_views_of_one_projection():
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V = 2, 140, 4, 2, 64, 64
    inp = synth.linattn_inputs(B, T, H, G, K, V, "bf16", 3)
    q, k, v, do = (dev(inp[x], "bf16") for x in ("q", "k", "v", "do"))
    wide = torch.cat([x.reshape(B, T, -1) for x in (q, k, v)], dim=-1)
    a, b, c = wide.split([G * K, G * K, H * V], dim=-1)
    views = a.view(B, T, G, K), b.view(B, T, G, K), c.view(B, T, H, V)
    la = dev(inp["log_decay"])
    o1, s1 = ssd.linattn_forward(q, k, v, la)
    o2, s2 = ssd.linattn_forward(*views, la)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    dop = torch.cat([do, do], dim=-2)[:, :, :H]  # strided over steps
    g1 = ssd.linattn_backward(q, k, v, la, None, do)
    g2 = ssd.linattn_backward(*views, la, None, dop)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_fp32_sums_keep_their_bits():
    """Rounding errors of fp32 products and sums are of either sign and add up as
    their squares do: an output's error stays at a few 2^-24 of the outputs'
    size however many terms it has.  Roundings of one direction (or operands
    of fewer bits) add up to tens of them over a thousand steps."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(2, 1024, 3, 3, 64, 64, "f32", 7, (-0.002, -0.004, -0.03))
    ro, rS = linattn.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["state0"], 1.0, None)
    o, S = ssd.linattn_forward(*(dev(inp[x]) for x in ("q", "k", "v", "log_decay", "state0")))
    for got, ref in ((host(o), ro), (host(S), rS)):
        err = np.sqrt(np.mean((got - ref) ** 2) / np.mean(ref ** 2))
        assert err <= 8 * 2.0 ** -24, err


def test_two_runs_are_equal_and_streams_are_followed():
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(2, 600, 4, 2, 64, 64, "bf16", 4)
    q, k, v, do = (dev(inp[x], "bf16") for x in ("q", "k", "v", "do"))
    la, s0, ds = dev(inp["log_decay"]), dev(inp["state0"]), dev(inp["dstate"])
    o, S = ssd.linattn_forward(q, k, v, la, s0)
    g = ssd.linattn_backward(q, k, v, la, s0, do, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, S2 = ssd.linattn_forward(q, k, v, la, s0, stream=side)
    g2 = ssd.linattn_backward(q, k, v, la, s0, do, ds, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("T", [100, 5000])
def test_the_state_in_place(T):
    """The final state written over the first one, rows whole and shared out."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    for dtype in ("bf16", "f32"):
        inp = synth.linattn_inputs(1, T, 2, 1, 64, 64, dtype, 8, (-0.01, -0.002))
        q, k, v = (dev(inp[x], dtype) for x in "qkv")
        la, s0 = dev(inp["log_decay"]), dev(inp["state0"])
        o, S = ssd.linattn_forward(q, k, v, la, s0.clone())
        o2, S2 = ssd.linattn_forward(q, k, v, la, s0, out={"state": s0})
        assert S2 is s0 and torch.equal(S, s0) and torch.equal(o, o2)


def test_a_row_alone_is_the_row_in_a_batch():
    """Rows are independent, whatever is in the others."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(3, 200, 2, 2, 64, 64, "bf16", 6)
    q, k, v = (dev(inp[x], "bf16") for x in "qkv")
    q[0] = float("nan")
    k[2] = float("inf")
    la = dev(inp["log_decay"])
    o, S = ssd.linattn_forward(q, k, v, la)
    o1, S1 = ssd.linattn_forward(q[1:2], k[1:2], v[1:2], la)
    ro, _ = linattn.forward(inp["q"][1:2], inp["k"][1:2], inp["v"][1:2], inp["log_decay"])
    mo, _ = linattn.forward(*(np.abs(inp[x][1:2]) for x in "qkv"), inp["log_decay"])
    for x in (o[1:2], o1):
        check(host(x), ro, mo, tol("bf16", 0))
    assert torch.isfinite(S[1]).all()


@pytest.mark.parametrize("case", [(1, 1, 1, 8, 8, "f32"), (3, 4, 2, 128, 64, "bf16"),
                                  (2, 6, 3, 80, 40, "bf16"), (5, 2, 2, 64, 128, "f32"),
                                  (2, 2, 1, 32, 16, "bf16"), (1, 3, 1, 16, 120, "f32"),
                                  # enough rows for the larger tiles
                                  (80, 4, 2, 80, 40, "bf16"), (64, 8, 1, 64, 24, "f32"),
                                  (160, 4, 4, 32, 72, "bf16"), (320, 2, 1, 16, 8, "f32")])
@pytest.mark.parametrize("rows", [False, True])
def test_step(case, rows):
    """One token: a state's element sees two rounded products and a sum, o a sum
    of K of them."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, H, G, K, V, dtype = case
    inp = synth.linattn_inputs(B, 1, H, G, K, V, dtype, 40, (-0.2, -np.inf, 0.0))
    la = inp["log_decay"]
    if rows:
        la = synth.round_to(np.log(np.random.default_rng(1).uniform(0.01, 1, (B, H))), "f32")
    q, k, v = (inp[x][:, 0] for x in "qkv")
    ro, rS = linattn.step(q, k, v, la, inp["state0"], 0.5)
    mo, mS = linattn.step(np.abs(q), np.abs(k), np.abs(v), la, np.abs(inp["state0"]), 0.5)
    s = dev(inp["state0"])
    keep = s.clone()
    o, S = ssd.linattn_step(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(la), s, scale=0.5)
    assert torch.equal(s, keep)
    check(host(S), rS, mS, 8 * 2.0 ** -24)
    check(host(o), ro, mo, (K + 16) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0))
    o2, S2 = ssd.linattn_step(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(la), s, scale=0.5,
                              state_out=s)
    assert S2 is s and torch.equal(s, S) and torch.equal(o, o2)


def test_step_slots():
    """Rows by slot; an idle row's output is zero and no state is touched."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(4, 1, 2, 1, 64, 64, "bf16", 41, (-0.2, -0.01))
    pool = torch.randn(6, 2, 64, 64, device="cuda")
    was = pool.clone()
    slots = torch.tensor([5, -1, 0, 6], dtype=torch.int32, device="cuda")
    q, k, v = (dev(inp[x][:, 0], "bf16") for x in "qkv")
    la = dev(inp["log_decay"])
    o, out = ssd.linattn_step(q, k, v, la, pool, slots=slots)
    assert out is pool
    ref_o, ref_s = ssd.linattn_step(q, k, v, la, torch.stack([was[5], was[1], was[0], was[2]]))
    assert torch.equal(o[0], ref_o[0]) and torch.equal(o[2], ref_o[2])
    assert not o[1].any() and not o[3].any()
    assert torch.equal(pool[5], ref_s[0]) and torch.equal(pool[0], ref_s[2])
    assert torch.equal(pool[1:5], was[1:5])


def test_steps_continue_a_prompt():
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.linattn_inputs(2, 140, 4, 2, 64, 64, "bf16", 42)
    q, k, v = (dev(inp[x], "bf16") for x in "qkv")
    la = dev(inp["log_decay"])
    o, S = ssd.linattn_forward(q, k, v, la)
    _, s = ssd.linattn_forward(q[:, :130], k[:, :130], v[:, :130], la)
    ro, rS = linattn.forward(inp["q"], inp["k"], inp["v"], inp["log_decay"])
    mo, mS = linattn.forward(*(np.abs(inp[x]) for x in "qkv"), inp["log_decay"])
    for t in range(130, 140):
        y, s = ssd.linattn_step(q[:, t], k[:, t], v[:, t], la, s, state_out=s)
        check(host(y), ro[:, t], mo[:, t], tol("bf16", 0))
    check(host(s), rS, mS, 2.0 ** -16)


def test_step_is_the_ssd_core_s_recurrence():
    """v = dt x, k = B, q = C, log_decay = dt A, o + D x: the core's last step."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    dims = synth.Dims(2, 48, 4, 64, 64, 2, 16, "f32")
    inp = synth.make_inputs(dims, 12, True, "softplus")
    t = {n: dev(inp[n]) for n in ("x", "dt", "A", "B", "C", "D", "h0")}
    y, final, hist = ssd.forward(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], chunk=16)
    _, s, _ = ssd.forward(*(t[n][:, :32].contiguous() if n in ("x", "dt", "B", "C") else t[n]
                            for n in ("x", "dt", "A", "B", "C", "D", "h0")), chunk=16)
    for i in range(32, 48):
        x, dt = t["x"][:, i], t["dt"][:, i]
        o, s = ssd.linattn_step(t["C"][:, i], t["B"][:, i], dt[..., None] * x, dt * t["A"], s)
    o = o + t["D"][None, :, None] * x
    # both sides are within the core's fp32 tolerance of the same recurrence
    assert float((s - final).abs().max() / final.abs().max()) <= 2e-4
    assert float((o - y[:, -1]).abs().max() / y[:, -1].abs().max()) <= 2e-4


def test_refusals():
    import torch
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, v, la = z(2, 5, 2, 16), z(2, 5, 4, 16), z(4)
    fwd = ssd.linattn_forward
    fwd(q, q, v, la)
    with pytest.raises(nat.SsdError):
        fwd(z(2, 5, 2, 12), z(2, 5, 2, 12), v, la)
    with pytest.raises(nat.SsdError):
        fwd(z(2, 5, 2, 136), z(2, 5, 2, 136), v, la)
    with pytest.raises(nat.SsdError):
        fwd(z(2, 5, 3, 16), z(2, 5, 3, 16), v, la)  # heads not a multiple of groups
    with pytest.raises(nat.SsdError):
        fwd(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 16), la)
    with pytest.raises(TypeError):
        fwd(q.half(), q.half(), v.half(), la)
    with pytest.raises(TypeError):
        fwd(q, q.bfloat16(), v, la)
    with pytest.raises(TypeError):
        fwd(q, q, v, la.double())
    with pytest.raises(TypeError):
        fwd(q, q, v, la, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        fwd(q, q, v, la, lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fwd(q, q, v, la[:2])
    with pytest.raises(ValueError):
        fwd(q.transpose(2, 3), q.transpose(2, 3), v, la)
    with pytest.raises(ValueError):
        fwd(q.cpu(), q.cpu(), v.cpu(), la.cpu())
    with pytest.raises(ValueError):
        fwd(q, q, v, la, z(2, 4, 16, 8))
    with pytest.raises(nat.SsdError):  # steps 34 floats apart
        wide = z(2, 5, 2 * 16 + 2)
        fwd(wide[:, :, :32].unflatten(2, (2, 16)), q, v, la)
    with pytest.raises(nat.SsdError):  # not on a 16-byte boundary
        flat = z(2 * 5 * 2 * 16 + 1)
        fwd(flat[1:].view(2, 5, 2, 16), q, v, la)
    with pytest.raises(nat.SsdError):
        fwd(q, q, v, la, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    st = z(2, 4, 16, 16)
    step = ssd.linattn_step
    step(q[:, 0], q[:, 0], v[:, 0], la, st)
    with pytest.raises(ValueError):
        step(q, q, v, la, st)
    with pytest.raises(ValueError):
        step(q[:, 0], q[:, 0], v[:, 0], la, st[:1])
    with pytest.raises(TypeError):
        step(q[:, 0], q[:, 0], v[:, 0], la, st, slots=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        ssd.linattn_backward(q, q, v, la, None, v[:1])
