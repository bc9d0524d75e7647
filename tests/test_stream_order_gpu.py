"""Calls on one stream read what the calls before them write, without a
synchronisation between them, wherever a kernel may start before the kernel
ahead of it has ended."""
import pytest

from state_space_model_analytic_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def core(T, seed):
    """Inputs of the core at a size whose state scans are fused (128 heads over
    all rows), as device tensors by name."""
    import torch
    inp = synth.make_inputs(synth.Dims(4, T, 32, 64, 128, 1, 256, "bf16"), seed, True, "softplus")
    t = {n: torch.from_numpy(inp[n]).float().cuda() for n in ("x", "dt", "A", "B", "C", "D", "h0", "dy")}
    for n in ("x", "B", "C", "dy"):
        t[n] = t[n].bfloat16()
    return t


def args(t, **other):
    return [other.get(n, t[n]) for n in ("x", "dt", "A", "B", "C", "D", "h0")]


@pytest.mark.parametrize("history", [False, True])
def test_two_layers_backward(history):
    """The upper layer's dx is the lower layer's dy."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    up, low = core(1024, 1), core(1024, 2)
    cs = [ssd.forward(*args(t), chunk=256)[2] if history else None for t in (up, low)]

    def chain(synchronise, dx):
        dx.fill_(7.0)
        g = ssd.backward(*args(up), up["dy"], cs[0], chunk=256, out={"dx": dx})
        if synchronise:
            torch.cuda.synchronize()
        return ssd.backward(*args(low), g["dx"], cs[1], chunk=256)

    dx = torch.empty_like(up["x"])
    want = chain(True, dx)
    for _ in range(5):
        got = chain(False, dx)
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("operand", ["x", "dy"])
def test_linear_attention_into_the_core(operand):
    """The output of a walk is an input of the core's backward, whose first
    kernel may start before the kernel ahead of it has ended."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    t = core(2048, 3)
    g = torch.Generator("cuda").manual_seed(4)
    q, k, v = (torch.randn(4, 2048, 32, d, generator=g, device="cuda").bfloat16() for d in (128, 128, 64))
    la = torch.full((32,), -0.05, device="cuda")

    def chain(synchronise, o):
        o.fill_(7.0)
        ssd.linattn_forward(q, k, v, la, scale=0.01, out={"o": o})
        if synchronise:
            torch.cuda.synchronize()
        return ssd.backward(*args(t, **{operand: o}), o if operand == "dy" else t["dy"], None, chunk=256)

    o = torch.empty_like(v)
    want = chain(True, o)
    for _ in range(5):
        got = chain(False, o)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_temporary_operands_on_another_stream():
    """An operand dropped on return is not handed out again while the other
    stream still has the call ahead of it."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    g = torch.Generator("cuda").manual_seed(6)
    q, k = (torch.randn(2, 300, 2, 64, generator=g, device="cuda") for _ in range(2))
    v = torch.randn(2, 300, 4, 64, generator=g, device="cuda")
    la = torch.full((4,), -0.05, device="cuda")
    grads = [torch.randn(n, generator=g, device="cuda") for n in (1000, 70001)]
    want = ssd.linattn_forward(q, k, v, la)
    want_n = ssd.clip_grad_norm(grads, 1.0, out=[torch.empty_like(t) for t in grads])
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(20):
            big.fill_(i)
    got = ssd.linattn_forward(q.clone(), k.clone(), v.clone(), la.clone(), stream=side)
    got_n = ssd.clip_grad_norm([t.clone() for t in grads], 1.0, stream=side)
    trash = [torch.full_like(t, float("nan")) for t in (q, k, v, la, *grads) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(got_n, want_n)
    del trash


def test_the_core_on_another_stream():
    """Dropped operands and the call's own workspace, behind a busy stream."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    t = core(512, 5)
    cs = ssd.forward(*args(t), chunk=256)[2]
    want = ssd.backward(*args(t), t["dy"], cs, chunk=256)
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(20):
            big.fill_(i)
    got = ssd.backward(*(a.clone() for a in args(t)), t["dy"].clone(), cs.clone(), chunk=256, stream=side)
    trash = [torch.full_like(a, float("nan")) for a in (*t.values(), cs) for _ in range(3)]
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    del trash
