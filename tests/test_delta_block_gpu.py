"""A layer of a delta-rule model as it is used: layer norm, projections, the delta rule
over unit keys, the gated RMS norm and the residual; trained through all of them, and
prompts continued token by token.

The same block in float64, by plain operations and torch's differentiation, from the
same (fp32) parameters; the block's own projections are fp32.  A value passes through
some ten operators, each within 2^-19 of its outputs' root mean square (what their own
tests hold them to), with gains below 4 between them, and the token steps and prompts
through the same ones: 2^-14 of the root mean square."""
import pytest

pytestmark = pytest.mark.gpu
B, T, H, G, K, V, WIDTH = 3, 90, 4, 2, 32, 64, 96
TOL = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def parameters():
    import torch
    gen = torch.Generator("cuda").manual_seed(3)
    r = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    return {"wn": 1 + r(WIDTH, std=0.1), "bn": r(WIDTH, std=0.1),
            "wq": r(WIDTH, G * K, std=0.1), "wk": r(WIDTH, G * K, std=0.1), "wv": r(WIDTH, H * V, std=0.1),
            "wa": r(WIDTH, H, std=0.1), "wb": r(WIDTH, H, std=0.1), "wz": r(WIDTH, H * V, std=0.1),
            "wg": 1 + r(H * V, std=0.1), "wo": r(H * V, WIDTH, std=0.1)}


def operators():
    """torch's differentiation through the library's operators."""
    import torch
    import state_space_model_analytic_gb300 as ssd

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, stats = ssd.layer_norm_forward(x, w, b, 1e-5)
            ctx.save_for_backward(x, w, stats)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, stats = ctx.saved_tensors
            g = ssd.layer_norm_backward(x, w, dy.contiguous(), 1e-5, stats)
            return g["dx"], g["dweight"], g["dbias"]

    class Delta(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, la, be, s0, lens):
            o, s = ssd.delta_rule_forward(q, k, v, la, be, s0, scale=K ** -0.5, lens=lens)
            ctx.save_for_backward(q, k, v, la, be, s0, lens)
            return o, s

        @staticmethod
        def backward(ctx, do, ds):
            *a, lens = ctx.saved_tensors
            g = ssd.delta_rule_backward(*a, do.contiguous(), ds.contiguous(), scale=K ** -0.5, lens=lens)
            return tuple(g[n] for n in ("dq", "dk", "dv", "dlog_decay", "dbeta", "dstate0")) + (None,)

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, z, w):
            o, inv = ssd.rmsnorm_gated_forward(y, z, w, 1e-5)
            ctx.save_for_backward(y, z, w, inv)
            return o

        @staticmethod
        def backward(ctx, dout):
            y, z, w, inv = ctx.saved_tensors
            g = ssd.rmsnorm_gated_backward(y, z, w, 1e-5, dout.contiguous(), inv)
            return g["dy"], g["dz"], g["dweight"]

    return Norm.apply, Delta.apply, Gated.apply


def block(x, s0, lens, p, norm, delta, gated):
    import torch
    n = norm(x, p["wn"], p["bn"])
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    q, k = (unit(torch.nn.functional.silu(n @ p[w]).unflatten(-1, (G, K))) for w in ("wq", "wk"))
    v = (n @ p["wv"]).unflatten(-1, (H, V))
    la, be = -torch.nn.functional.softplus(n @ p["wa"] - 2), torch.sigmoid(n @ p["wb"])
    o, s = delta(q.contiguous(), k.contiguous(), v.contiguous(), la.contiguous(), be.contiguous(), s0, lens)
    return x + gated(o.flatten(-2), (n @ p["wz"]).contiguous(), p["wg"]) @ p["wo"], s


def plain():
    import torch

    def norm(x, w, b):
        d = x - x.mean(-1, keepdim=True)
        return d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def delta(q, k, v, la, be, s0, lens):
        q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
        S, o = s0, []
        for t in range(q.shape[1]):
            n = torch.full((B,), T, device="cuda") if lens is None else lens
            live = (t < n)[:, None, None, None]
            A = la[:, t].exp()[..., None, None] * S
            e = v[:, t] - (A @ k[:, t][..., None])[..., 0]
            S = torch.where(live, A + (be[:, t][..., None] * e)[..., None] * k[:, t][..., None, :], S)
            y = (S @ q[:, t][..., None])[..., 0] * K ** -0.5
            o.append(torch.where(live[..., 0], y, 0.0))
        return torch.stack(o, 1), S

    def gated(y, z, w):
        n = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        return n * w * torch.nn.functional.silu(z)
    return norm, delta, gated


def inputs():
    import torch
    gen = torch.Generator("cuda").manual_seed(4)
    return (torch.randn(B, T, WIDTH, generator=gen, device="cuda"),
            torch.randn(B, H, V, K, generator=gen, device="cuda") * 0.5)


def close(got, want):
    err = (got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()
    assert float(err) <= TOL, float(err)


@pytest.mark.parametrize("lens", [None, (90, 0, 41)])
def test_a_layer_and_its_gradients(lens):
    import torch
    x, s0 = inputs()
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(6)
    results = []
    for ops, dt in ((operators(), torch.float32), (plain(), torch.float64)):
        p = {n: t.to(dt).requires_grad_() for n, t in parameters().items()}
        xs, ss = x.to(dt).requires_grad_(), s0.to(dt).requires_grad_()
        y, s = block(xs, ss, ln, p, *ops)
        if not results:
            wy, ws = torch.randn(y.shape, generator=gen, device="cuda"), torch.randn(
                s.shape, generator=gen, device="cuda")
        g = torch.autograd.grad((y * wy.to(dt)).sum() + (s * ws.to(dt)).sum(),
                                [xs, ss, *p.values()])
        results.append([y.detach(), s.detach(), *g])
    for got, want in zip(*results):
        close(got, want)


def test_a_prompt_continued_token_by_token():
    """The layer over 90 steps, and over 80 with ten single tokens behind them."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    x, s0 = inputs()
    p = parameters()
    norm, delta, gated = operators()
    y, s = block(x, s0, None, p, norm, delta, gated)
    y1, state = block(x[:, :80].contiguous(), s0, None, p, norm, delta, gated)
    close(y1, y[:, :80].double())

    def one(q, k, v, la, be, state, _):
        a = [t[:, 0].contiguous() for t in (q, k, v, la, be)]
        o, new = ssd.delta_rule_step(*a, state, scale=K ** -0.5)
        return o[:, None], new

    for t in range(80, 90):
        yt, state = block(x[:, t:t + 1].contiguous(), state, None, p, norm, one, gated)
        close(yt, y[:, t:t + 1].double())
    close(state, s.double())
