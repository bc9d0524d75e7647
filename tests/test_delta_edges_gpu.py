"""GPU tests of the gated delta rule and the layer norm where the first parity tests do
not reach: every number of warps that share a state's rows, operands scaled by powers
of two, values that are not finite, offsets past 32 bits, several calls at once.

The rule does not change when a step's k and v are multiplied by 2^m and its beta by
2^-2m, and it is linear in q, v and the state.  No sum, split or rounding depends on
such a factor, so those results are compared bit for bit."""
import numpy as np
import pytest

from oracle import delta
from state_space_model_analytic_gb300 import synth
from test_parity_delta_gpu import NAMES, _built, check, dev, host, on_device, operands, rounded  # noqa: F401

pytestmark = pytest.mark.gpu


# o = e^g H q + P U takes H, P and U in 11 bits where it is bf16: H off by 2^-12, a term of
# P U by twice that, and the reference's size is |q| times the sum of the terms'
# magnitudes, so o is off by 2^-11 size at most.  (With many terms of any sign it is far
# less: 2^-15 where keys are long.)
O_OF_SIZE = 2.0 ** -11


# B, T, H, G, K, V, dtype, lens: CTAs of 64, 32 or 16 columns of v, as many warps a row
SHARES = [
    (2, 100, 36, 4, 128, 64, "bf16", None),              # 144 CTAs with two warps a row
    (2, 100, 36, 36, 64, 40, "bf16", (100, 65)),         # (the second CTA of a head half empty)
    (2, 70, 30, 6, 128, 72, "f32", None),                # three CTAs a head, the last of 8 columns
    (4, 100, 40, 8, 128, 64, "bf16", (100, 64, 63, 1)),  # more than there are SMs: one warp a row
    (4, 100, 40, 8, 128, 24, "bf16", None),              # and warps without columns
    (4, 70, 40, 40, 64, 24, "f32", (0, 70, 32, 33)),
    (3, 40, 60, 20, 128, 64, "f32", None),
    # rows of any length in any order, as many as are put in order and more
    (256, 40, 1, 1, 16, 8, "bf16", tuple(i * 7 % 41 for i in range(256))),
    (300, 40, 1, 1, 16, 8, "f32", tuple(i * 7 % 41 for i in range(300))),
    (40, 130, 8, 2, 128, 16, "bf16", tuple(i * 37 % 131 for i in range(40))),
]


@pytest.mark.parametrize("case", SHARES, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_warps_that_share_rows(case):
    import state_space_model_analytic_gb300 as ssd
    B, T, H, G, K, V, dtype, lens = case
    inp = synth.delta_inputs(B, T, H, G, K, V, dtype, 60)
    x, s0 = operands(inp, dtype, lens), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0, scale=0.5, lens=on_device(lens))
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES), inp["state0"], 0.5, lens)
    check(host(o), ro, mo, T, rounded(dtype), O_OF_SIZE if dtype == "bf16" else 0.0)
    check(host(S), rS, mS, T)
    g = ssd.delta_rule_backward(*x, s0, dev(inp["do"], dtype), dev(inp["dstate"]), scale=0.5,
                                lens=on_device(lens))
    ref, size = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"], 0.5,
                               lens)
    for n in ref:
        check(host(g[n]), ref[n], size[n], T, rounded(dtype) if n in ("dq", "dk", "dv") else 0.0)


@pytest.mark.parametrize("H", [2, 80])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_powers_of_two(dtype, H):
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, K, V = 2, 150, 64, 64
    inp = synth.delta_inputs(B, T, H, H, K, V, dtype, 61)
    rng = np.random.default_rng(62)
    two = lambda lo, hi: torch.from_numpy(np.exp2(rng.integers(lo, hi, (B, T, H)))).float().cuda()  # noqa: E731
    fk, fq = two(-20, 21), two(-10, 11)
    q, k, v, la, be = operands(inp, dtype)
    s0, do, ds = dev(inp["state0"]), dev(inp["do"], dtype), dev(inp["dstate"])
    t = lambda x, f: (x.float() * f[..., None]).to(x.dtype)  # noqa: E731
    o, S = ssd.delta_rule_forward(q, k, v, la, be, s0)
    o2, S2 = ssd.delta_rule_forward(t(q, fq), t(k, fk), t(v, fk), la, be / (fk * fk), s0)
    assert torch.equal(t(o, fq), o2) and torch.equal(S, S2)
    g = ssd.delta_rule_backward(q, k, v, la, be, s0, do, ds)
    h = ssd.delta_rule_backward(t(q, fq), t(k, fk), t(v, fk), la, be / (fk * fk), s0, t(do, 1 / fq), ds)
    assert torch.equal(t(g["dq"], 1 / fq), h["dq"])
    assert torch.equal(t(g["dk"], 1 / fk), h["dk"]) and torch.equal(t(g["dv"], 1 / fk), h["dv"])
    assert torch.equal(g["dlog_decay"], h["dlog_decay"])
    assert torch.equal(g["dbeta"] * fk * fk, h["dbeta"]) and torch.equal(g["dstate0"], h["dstate0"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("f", [2.0 ** 60, 2.0 ** -60])
def test_large_and_small_values(f, dtype):
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 150, 2, 1, 128, 64, dtype, 63)
    q, k, v, la, be = operands(inp, dtype)
    s0, do, ds = dev(inp["state0"]), dev(inp["do"], dtype), dev(inp["dstate"])
    o, S = ssd.delta_rule_forward(q, k, v, la, be, s0)
    o2, S2 = ssd.delta_rule_forward(q, k, v * f, la, be, s0 * f)
    assert torch.equal(o * f, o2) and torch.equal(S * f, S2)
    g = ssd.delta_rule_backward(q, k, v, la, be, s0, do, ds)
    h = ssd.delta_rule_backward(q, k, v * f, la, be, s0 * f, do * (1 / f), ds * (1 / f))
    for n in ("dq", "dk", "dlog_decay", "dbeta"):
        assert torch.equal(g[n], h[n]), n
    assert torch.equal(g["dv"] * (1 / f), h["dv"]) and torch.equal(g["dstate0"] * (1 / f), h["dstate0"])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_value_stays_in_its_column(dtype, bad):
    """Columns of v are independent of one another, and steps of those after them (of
    the same chunk's steps before it that is not promised)."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 200, 2, 1, 64, 64, dtype, 64)
    x = operands(inp, dtype)
    o, S = ssd.delta_rule_forward(*x)
    x[2][0, 70, 1, 5] = bad
    o2, S2 = ssd.delta_rule_forward(*x)
    assert not torch.isfinite(o2[0, 70:, 1, 5]).any() and not torch.isfinite(S2[0, 1, 5]).any()
    assert torch.equal(o2[0, :64, 1, 5], o[0, :64, 1, 5])
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[0, :, 1, 5] = False
    assert torch.equal(o2[keep], o[keep])
    keep = torch.ones_like(S, dtype=torch.bool)
    keep[0, 1, 5] = False
    assert torch.equal(S2[keep], S[keep])


def test_write_strengths_of_any_sign():
    """beta zero (nothing is written), negative, and two (reflections)."""
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(2, 150, 4, 2, 64, 64, "f32", 65)
    k = inp["k"]
    inp["k"] = synth.round_to(k / np.sqrt((k * k).sum(-1, keepdims=True)), "f32")
    inp["beta"] = np.broadcast_to(np.array([0.0, -0.1, 2.0, 1.0]), inp["beta"].shape).copy()
    x, s0 = operands(inp, "f32"), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0)
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES), inp["state0"])
    check(host(o), ro, mo, 150)
    check(host(S), rS, mS, 150)
    g = ssd.delta_rule_backward(*x, s0, dev(inp["do"]), dev(inp["dstate"]))
    ref, size = delta.backward(*(inp[n] for n in NAMES), inp["state0"], inp["do"], inp["dstate"])
    for n in ref:
        check(host(g[n]), ref[n], size[n], 150)


@pytest.mark.parametrize("strengths", [(0.0, -0.1, 2.0, 1.0), (1.0, 1.0, 1.0, 40.0)],
                         ids=["signs", "once_large"])
def test_alike_keys_of_many_heads(strengths):
    """Keys that hardly differ, 160 (row, head) pairs of 128 columns; the last strength
    of a head in one step alone, which multiplies the memory by 1 - 40.

    (The steps 75 and 76 write 40 times what others do, and of opposite sign, so what o
    is rounded by does not average out.)"""
    import state_space_model_analytic_gb300 as ssd
    B, T, H, K = 2, 130, 80, 128
    inp = synth.delta_inputs(B, T, H, H, K, 32, "bf16", 71)
    k = 1.0 + 0.05 * inp["k"]
    inp["k"] = synth.round_to(k / np.sqrt((k * k).sum(-1, keepdims=True)), "bf16")
    be = np.ones_like(inp["beta"])
    be[:, :, 0::2], be[:, :, 1::2] = strengths[0], strengths[1]
    be[:, ::3, 1::2] = strengths[2]
    be[:, 75] = strengths[3]
    inp["beta"] = be
    x, s0 = operands(inp, "bf16"), dev(inp["state0"])
    o, S = ssd.delta_rule_forward(*x, s0)
    ro, rS, mo, mS = delta.forward(*(inp[n] for n in NAMES), inp["state0"])
    check(host(o), ro, mo, T, 2.0 ** -8, O_OF_SIZE)
    check(host(S), rS, mS, T)


def test_operands_shared_by_all_rows_are_refused():
    """Views whose rows are the same memory (a batch stride of zero)."""
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    inp = synth.delta_inputs(3, 100, 4, 2, 64, 64, "bf16", 66)
    q, k, v, la, be = operands(inp, "bf16")
    with pytest.raises(nat.SsdError):
        ssd.delta_rule_forward(q[:1].expand(3, -1, -1, -1), k, v, la, be)
    with pytest.raises(nat.SsdError):
        ssd.delta_rule_backward(q, k, v, la, be, None, v[:1].expand(3, -1, -1, -1))


@pytest.mark.parametrize("dim", ["batch", "step"])
def test_offsets_past_32_bits(dim):
    import torch
    import state_space_model_analytic_gb300 as ssd
    B, T, H, K = (2, 70, 2, 64) if dim == "batch" else (1, 4, 2, 64)
    inp = synth.delta_inputs(B, T, H, H, K, K, "bf16", 67)
    x, do = operands(inp, "bf16"), dev(inp["do"], "bf16")
    far = 2 ** 31 + 4096 if dim == "batch" else 2 ** 30 + 4096
    pool = torch.empty(4 * 2 ** 30, dtype=torch.bfloat16, device="cuda")
    strides = (far, 4 * H * K, K, 1) if dim == "batch" else (0, far, K, 1)
    views = []
    for i, t in enumerate((*x[:3], do)):
        w = pool.as_strided((B, T, H, K), strides, i * H * K)
        w.copy_(t)
        views.append(w)
    if dim == "step":
        assert (T - 1) * far + 4 * H * K <= pool.numel()
    for a, b in zip(ssd.delta_rule_forward(*x), ssd.delta_rule_forward(*views[:3], *x[3:])):
        assert torch.equal(a, b)
    g = ssd.delta_rule_backward(*x, None, do)
    h = ssd.delta_rule_backward(*views[:3], *x[3:], None, views[3])
    assert all(torch.equal(g[n], h[n]) for n in g)
    w = torch.randn(H * K, device="cuda")
    rows = pool.as_strided((4, H * K), (2 ** 30 + 4096, 1))
    rows.copy_(torch.randn(4, H * K))
    y, st = ssd.layer_norm_forward(rows, w, w, 1e-5)
    z, _ = ssd.layer_norm_forward(rows.contiguous(), w, w, 1e-5)
    assert torch.equal(y, z)
    dy = torch.randn(4, H * K, device="cuda").bfloat16()
    a, b = (ssd.layer_norm_backward(t, w, dy, 1e-5, st) for t in (rows, rows.contiguous()))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_many_rows_of_one_token():
    import torch
    import state_space_model_analytic_gb300 as ssd
    inp = synth.delta_inputs(5, 1, 1, 1, 8, 8, "f32", 68)
    x = [t[:, 0].repeat(13107, *[1] * (t.dim() - 2)).contiguous() for t in operands(inp, "f32")]
    s = dev(inp["state0"])
    o, S = ssd.delta_rule_step(*x, s.repeat(13107, 1, 1, 1))
    ro, rS = ssd.delta_rule_step(*(t[:5].contiguous() for t in x), s)
    assert torch.equal(o.view(13107, 5, 1, 8), ro.expand(13107, -1, -1, -1))
    assert torch.equal(S.view(13107, 5, 1, 8, 8), rS.expand(13107, -1, -1, -1, -1))


def test_two_calls_at_once():
    """Forwards, gradients and norms on two streams at the same time."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    sets = []
    for seed in (69, 70):
        inp = synth.delta_inputs(2, 700, 8, 2, 128, 64, "bf16", seed)
        x, do = operands(inp, "bf16"), dev(inp["do"], "bf16")
        y = torch.randn(500, 768, device="cuda").bfloat16()
        sets.append((x, do, y, torch.randn(768, device="cuda")))

    def run(x, do, y, w, stream=None):
        o, S = ssd.delta_rule_forward(*x, stream=stream)
        g = ssd.delta_rule_backward(*x, None, do, stream=stream)
        n, st = ssd.layer_norm_forward(y, w, w, 1e-5, stream=stream)
        h = ssd.layer_norm_backward(y, w, n, 1e-5, st, stream=stream)
        return [o, S, *(g[k] for k in sorted(g)), n, *(h[k] for k in sorted(h))]

    alone = [run(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        both = [run(*s, stream=st) for s, st in zip(sets, streams)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(alone, both):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_captured_norm(dtype):
    """A norm and its gradients in a CUDA graph, replayed twice on other inputs; a
    second graph holds the same workspace."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    new = lambda *s: torch.randn(*s, device="cuda").to(kind)  # noqa: E731
    x, dy, w = new(700, 640), new(700, 640), torch.randn(640, device="cuda")
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")

    def run():
        y, st = ssd.layer_norm_forward(x, w, w, 1e-5)
        return y, ssd.layer_norm_backward(x, w, dy, 1e-5, st, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        graphs.append((graph, got))
    for _ in range(2):
        x.copy_(new(700, 640))
        dy.copy_(new(700, 640))
        for graph, _ in graphs:
            graph.replay()
        ry, rg = run()
        for _, (y, g) in graphs:
            assert torch.equal(y, ry) and all(torch.equal(g[n], rg[n]) for n in rg)
