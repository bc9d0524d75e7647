"""GPU parity of the gated delta rule (forward, gradients, single token) against the
float64 reference.

Tolerances.  The reference gives the size that an output's errors go by (products
of norms).  Operands held in 32 bits keep 22 bits in products, 2^-21 of each, whose
sums pass through at most 8 terms x 3 products of parts that the matrix instructions
round toward zero, 2^-23 of the sum each: 32 * 2^-23 a product in all, below 2^-17;
three products follow one another in a chunk and the chunks of a row add up, 32 steps
each at least: |error| <= 2^-16 max(1, T / 32) size.  A bf16 output is rounded by 2^-8
of itself; o takes the state and P in 11 bits, 2^-12 of each term, which as signs
differ is far less of o's size, the sum of its terms' magnitudes: 2^-15."""
import numpy as np
import pytest

from oracle import delta
from state_space_model_analytic_gb300 import synth

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "log_decay", "beta")


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


def operands(inp, dtype, lens=None):
    return [dev(poison(inp[n], lens), dtype if n in "qkv" else "f32") for n in NAMES]


def on_device(lens):
    import torch
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(got, ref, size, T, rounded=0.0, of_size=0.0):
    assert got.shape == ref.shape and np.isfinite(got).all()
    t = 2.0 ** -16 * max(1.0, T / 32)
    err, most = np.abs(got - ref), (t + of_size) * size + (rounded + 2.0 ** -23) * np.abs(ref) + 1e-30
    bad = err > most
    assert not bad.any(), (int(bad.sum()), bad.size, float((err / most).max()))


def rounded(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0


# B, T, H, G, K, V, dtype, lens, decays
CASES = [
    (1, 1, 1, 1, 8, 8, "f32", None, None),
    (2, 3, 2, 1, 16, 8, "bf16", None, None),
    (2, 31, 4, 2, 16, 24, "f32", None, (-0.5, 0.0)),
    (1, 64, 2, 2, 64, 64, "bf16", None, None),
    (2, 65, 3, 3, 64, 64, "bf16", None, (-0.02, -3.0, -40.0, 0.0)),
    (1, 200, 4, 1, 128, 64, "bf16", None, None),
    (2, 130, 2, 2, 64, 128, "bf16", None, None),
    (1, 191, 2, 1, 128, 128, "bf16", None, (-0.01, -0.2)),
    (2, 200, 2, 2, 80, 40, "bf16", None, None),
    (1, 129, 2, 2, 72, 104, "bf16", None, None),
    (2, 77, 2, 2, 128, 128, "f32", None, None),
    (1, 320, 2, 2, 64, 64, "f32", None, (-0.003, -1.0, -0.1)),
    (5, 260, 2, 1, 64, 64, "bf16", (0, 1, 128, 259, 260), None),
    (4, 150, 4, 2, 128, 64, "bf16", (150, 129, 0, 2), (0.0, -0.1, -np.inf, -1e30, -0.3)),
    (3, 70, 2, 2, 32, 16, "f32", (70, 0, 33), (-np.inf, -0.2, -0.1)),
    (3, 190, 4, 2, 80, 40, "f32", (190, 65, 129), (-0.01, -0.4, -5.0, 0.0)),
    (1, 100, 1, 1, 24, 72, "f32", None, None),
    # more (row, head) pairs than SMs
    (16, 140, 12, 4, 64, 16, "bf16", None, None),
]
ids = [f"b{c[0]}t{c[1]}h{c[2]}g{c[3]}k{c[4]}v{c[5]}{c[6]}{'lens' if c[7] else ''}" for c in CASES]


def inputs(case):
    B, T, H, G, K, V, dtype, lens, decays = case
    return synth.delta_inputs(B, T, H, G, K, V, dtype, 100 + T, decays)


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case, with_state):
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, dtype, lens, _ = case
    inp = inputs(case)
    s0 = inp["state0"] if with_state else None
    o, S = ssd.delta_rule_forward(*operands(inp, dtype, lens), None if s0 is None else dev(s0),
                                  scale=0.25, lens=on_device(lens))
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES), s0, 0.25, lens)
    check(host(o), ro, mo, T, rounded(dtype), 2.0 ** -15)
    check(host(S), rS, mS, T)
    if lens is not None:
        for b, n in enumerate(lens):
            assert not o[b, n:].any()


@pytest.mark.parametrize("with_state", [False, True])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case, with_state):
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, dtype, lens, _ = case
    inp = inputs(case)
    s0, ds = (inp["state0"], inp["dstate"]) if with_state else (None, None)
    g = ssd.delta_rule_backward(*operands(inp, dtype, lens), None if s0 is None else dev(s0),
                                dev(poison(inp["do"], lens), dtype), None if ds is None else dev(ds),
                                scale=0.25, lens=on_device(lens))
    ref, size = delta.backward(*(inp[n] for n in NAMES), s0, inp["do"], ds, 0.25, lens)
    for n in ref:
        check(host(g[n]), ref[n], size[n], T, rounded(dtype) if n in ("dq", "dk", "dv") else 0.0)
    if lens is not None:
        for b, n in enumerate(lens):
            assert not any(g[x][b, n:].any() for x in g if x != "dstate0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_is_the_forward_s_difference(dtype):
    """Along a direction u of all inputs, the fp32 forward's difference quotient
    (fourth order: h^4 = 2^-24 of the loss's fifth derivative) against the sum of
    gradients times u.  The forward's own errors, 2^-20 of the loss's terms over h,
    are 2^-14 of them."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 150, 2, 1, 64, 64, "f32", 9)
    u = synth.delta_inputs(1, 150, 2, 1, 64, 64, "f32", 10)
    names = NAMES + ("state0",)
    u = {n: u[n] * 0.1 for n in names}

    def loss(h):
        o, S = ssd.delta_rule_forward(*(dev(inp[n] + h * u[n]) for n in names), scale=0.125)
        return float((host(o) * inp["do"]).sum() + (host(S) * inp["dstate"]).sum())

    h = 2.0 ** -6
    num = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    g = ssd.delta_rule_backward(*operands(inp, dtype), dev(inp["state0"]), dev(inp["do"], dtype),
                                dev(inp["dstate"]), scale=0.125)
    terms = [(host(g["d" + n]) * u[n]) for n in names]
    scale = np.sqrt(sum((t ** 2).sum() for t in terms))
    # bf16: the inputs' and outputs' own roundings, 2^-8 each of five factors at most
    assert abs(sum(t.sum() for t in terms) - num) <= (2.0 ** -5 if dtype == "bf16" else 2.0 ** -7) * scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_keep_their_bits(dtype):
    """An output's error stays at a few 2^-22 of the outputs' size over many chunks: a
    product's sums pass through 24 truncations of 2^-24 on average at most.  The terms
    of dlog_decay cancel to a thirtieth and less of their size."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(1, 1024, 3, 3, 64, 64, dtype, 7)
    ro, rS, _, _ = delta.forward(*(inp[n] for n in NAMES), inp["state0"], 1.0, None)
    x = operands(inp, dtype)
    o, S = ssd.delta_rule_forward(*x, dev(inp["state0"]))
    g = ssd.delta_rule_backward(*x, dev(inp["state0"]), dev(inp["do"], dtype), dev(inp["dstate"]))
    ref, _ = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    ref.update(o=ro, state=rS)
    g.update(o=o, state=S)
    most = {"o": 0.0018, "dq": 0.0018, "dk": 0.0018, "dv": 0.0018} if dtype == "bf16" else {}
    for n in ref:
        err = np.sqrt(np.mean((host(g[n]) - ref[n]) ** 2) / np.mean(ref[n] ** 2))
        assert err <= most.get(n, 2.0 ** (-17 if n == "dlog_decay" else -19)), (n, err)


def test_alike_keys():
    """Keys that hardly differ: (I + L beta)^-1 by powers of L would lose every digit."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 192, 2, 2, 64, 64, "bf16", 11)
    k = 1.0 + 0.05 * inp["k"]
    inp["k"] = synth.round_to(k / np.sqrt((k * k).sum(-1, keepdims=True)), "bf16")
    inp["beta"] = np.ones_like(inp["beta"])
    inp["log_decay"] = np.zeros_like(inp["log_decay"])
    x = operands(inp, "bf16")
    o, S = ssd.delta_rule_forward(*x, dev(inp["state0"]))
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES), inp["state0"])
    check(host(o), ro, mo, 192, 2.0 ** -8, 2.0 ** -15)
    check(host(S), rS, mS, 192)
    g = ssd.delta_rule_backward(*x, dev(inp["state0"]), dev(inp["do"], "bf16"), dev(inp["dstate"]))
    ref, size = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    for n in ref:
        check(host(g[n]), ref[n], size[n], 192, 2.0 ** -8 if n in ("dq", "dk", "dv") else 0.0)


def test_views_of_one_projection():
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V = 2, 140, 4, 2, 64, 64
    inp = synth.delta_inputs(B, T, H, G, K, V, "bf16", 3)
    q, k, v, la, be = operands(inp, "bf16")
    do = dev(inp["do"], "bf16")
    wide = torch.cat([x.reshape(B, T, -1) for x in (q, k, v)], dim=-1)
    a, b, c = wide.split([G * K, G * K, H * V], dim=-1)
    views = a.view(B, T, G, K), b.view(B, T, G, K), c.view(B, T, H, V)
    o1, s1 = ssd.delta_rule_forward(q, k, v, la, be)
    o2, s2 = ssd.delta_rule_forward(*views, la, be)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)
    dop = torch.cat([do, do], dim=-2)[:, :, :H]  # strided over steps
    g1 = ssd.delta_rule_backward(q, k, v, la, be, None, do)
    g2 = ssd.delta_rule_backward(*views, la, be, None, dop)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_two_runs_are_equal_and_streams_are_followed():
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 300, 4, 2, 64, 64, "bf16", 4)
    x = operands(inp, "bf16")
    do, s0, ds = dev(inp["do"], "bf16"), dev(inp["state0"]), dev(inp["dstate"])
    o, S = ssd.delta_rule_forward(*x, s0)
    g = ssd.delta_rule_backward(*x, s0, do, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, S2 = ssd.delta_rule_forward(*x, s0, stream=side)
    g2 = ssd.delta_rule_backward(*x, s0, do, ds, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_state_in_place(dtype):
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 100, 2, 1, 64, 96, dtype, 8)
    x, s0 = operands(inp, dtype), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0.clone())
    o2, S2 = ssd.delta_rule_forward(*x, s0, out={"state": s0})
    assert S2 is s0 and torch.equal(S, s0) and torch.equal(o, o2)


def test_a_row_alone_is_the_row_in_a_batch():
    """Rows are independent, whatever is in the others."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(3, 200, 2, 2, 64, 64, "bf16", 6)
    q, k, v, la, be = operands(inp, "bf16")
    q[0] = float("nan")
    k[2] = float("inf")
    o, S = ssd.delta_rule_forward(q, k, v, la, be)
    o1, S1 = ssd.delta_rule_forward(*(x[1:2] for x in (q, k, v, la, be)))
    assert torch.equal(o[1:2], o1) and torch.equal(S[1:2], S1) and torch.isfinite(o1).all()


def test_captured_and_replayed():
    """A forward and a backward in a CUDA graph, replayed on other inputs."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    a, b = (synth.delta_inputs(2, 130, 4, 2, 64, 64, "bf16", s) for s in (20, 21))
    x, do = operands(a, "bf16"), dev(a["do"], "bf16")
    ws = torch.empty(ssd.delta_rule_workspace_bytes(*x, backward=True), dtype=torch.uint8, device="cuda")
    run = lambda: (ssd.delta_rule_forward(*x), ssd.delta_rule_backward(*x, None, do, workspace=ws))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (o, S), g = run()
    y = operands(b, "bf16")
    for t, f in zip(x, y):
        t.copy_(f)
    do.copy_(dev(b["do"], "bf16"))
    graph.replay()
    ro, rS = ssd.delta_rule_forward(*y)
    rg = ssd.delta_rule_backward(*y, None, do)
    assert torch.equal(o, ro) and torch.equal(S, rS)
    assert all(torch.equal(g[n], rg[n]) for n in rg)


@pytest.mark.parametrize("case", [(1, 1, 1, 8, 8, "f32"), (3, 4, 2, 128, 64, "bf16"),
                                  (2, 6, 3, 80, 40, "bf16"), (5, 2, 2, 64, 128, "f32"),
                                  (2, 2, 1, 32, 16, "bf16"), (1, 3, 1, 16, 120, "f32"),
                                  # enough rows for the larger tiles
                                  (80, 4, 2, 80, 40, "bf16"), (64, 8, 1, 64, 24, "f32"),
                                  (160, 4, 4, 32, 72, "bf16"), (320, 2, 1, 16, 8, "f32")])
def test_step(case):
    """One token: dots of K rounded terms and their sums."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, H, G, K, V, dtype = case
    inp = synth.delta_inputs(B, 1, H, G, K, V, dtype, 40, (-0.2, -np.inf, 0.0, -0.01))
    x = [t[:, 0].contiguous() for t in operands(inp, dtype)]
    ro, rS = delta.step(*(inp[n][:, 0] for n in NAMES), inp["state0"], 0.5)
    _, _, mo, mS = delta.forward(*(inp[n] for n in NAMES), inp["state0"], 0.5)
    s = dev(inp["state0"])
    keep = s.clone()
    o, S = ssd.delta_rule_step(*x, s, scale=0.5)
    assert torch.equal(s, keep)
    n = (K + 16) * 2.0 ** -24
    assert (np.abs(host(S) - rS) <= n * mS + 1e-30).all()
    assert (np.abs(host(o) - ro) <= 2 * n * mo[:, 0] + rounded(dtype) * np.abs(ro) + 1e-30).all()
    o2, S2 = ssd.delta_rule_step(*x, s, scale=0.5, state_out=s)
    assert S2 is s and torch.equal(s, S) and torch.equal(o, o2)


def test_step_slots():
    """Rows by slot; an idle row's output is zero and no state is touched."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(4, 1, 2, 1, 64, 64, "bf16", 41)
    pool = torch.randn(6, 2, 64, 64, device="cuda")
    was = pool.clone()
    slots = torch.tensor([5, -1, 0, 6], dtype=torch.int32, device="cuda")
    x = [t[:, 0].contiguous() for t in operands(inp, "bf16")]
    o, out = ssd.delta_rule_step(*x, pool, slots=slots)
    assert out is pool
    ref_o, ref_s = ssd.delta_rule_step(*x, torch.stack([was[5], was[1], was[0], was[2]]))
    assert torch.equal(o[0], ref_o[0]) and torch.equal(o[2], ref_o[2])
    assert not o[1].any() and not o[3].any()
    assert torch.equal(pool[5], ref_s[0]) and torch.equal(pool[0], ref_s[2])
    assert torch.equal(pool[1:5], was[1:5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_continue_a_prompt(dtype):
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 140, 4, 2, 64, 64, dtype, 42)
    x = operands(inp, dtype)
    _, s = ssd.delta_rule_forward(*(t[:, :130].contiguous() for t in x))
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES))
    for t in range(130, 140):
        y, s = ssd.delta_rule_step(*(z[:, t].contiguous() for z in x), s, state_out=s)
        check(host(y), ro[:, t], mo[:, t], 140, rounded(dtype))
    check(host(s), rS, mS, 140)


def test_refusals():
    import torch
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    q, v, la = z(2, 5, 2, 16), z(2, 5, 4, 16), z(2, 5, 4)
    fwd = ssd.delta_rule_forward
    fwd(q, q, v, la, la)
    with pytest.raises(nat.SsdError):
        fwd(z(2, 5, 2, 12), z(2, 5, 2, 12), v, la, la)
    with pytest.raises(nat.SsdError):
        fwd(z(2, 5, 3, 16), z(2, 5, 3, 16), v, la, la)  # heads not a multiple of groups
    with pytest.raises(nat.SsdError):
        fwd(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 16), z(2, 0, 4), z(2, 0, 4))
    with pytest.raises(TypeError):
        fwd(q.half(), q.half(), v.half(), la, la)
    with pytest.raises(TypeError):
        fwd(q, q, v, la.double(), la)
    with pytest.raises(TypeError):
        fwd(q, q, v, la, la.bfloat16())
    with pytest.raises(ValueError):
        fwd(q, q, v, la[0, 0], la)
    with pytest.raises(ValueError):
        fwd(q, q, v, la, la[:, :4])
    with pytest.raises(ValueError):  # gates are dense
        fwd(q, q, v, la.transpose(0, 1).contiguous().transpose(0, 1), la)
    with pytest.raises(ValueError):
        fwd(q, q, v, la, la, z(2, 4, 16, 8))
    with pytest.raises(ValueError):
        ssd.delta_rule_backward(q, q, v, la, la, None, v[:1])
    with pytest.raises(nat.SsdError):
        ssd.delta_rule_backward(q, q, v, la, la, None, v,
                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ssd.delta_rule_backward(q, q, v, la, la, None, v, out={"dbeta": z(2, 5)})
    st = z(2, 4, 16, 16)
    step = ssd.delta_rule_step
    x = q[:, 0].contiguous(), q[:, 0].contiguous(), v[:, 0].contiguous(), la[:, 0].contiguous()
    step(*x, x[3], st)
    with pytest.raises(ValueError):
        step(*x, z(4), st)
    with pytest.raises(ValueError):
        step(*x, x[3], st[:1])
    with pytest.raises(TypeError):
        step(*x, x[3], st, slots=torch.zeros(2, device="cuda"))
