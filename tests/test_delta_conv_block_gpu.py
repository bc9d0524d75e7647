"""The delta-rule layer with its short convolution: layer norm, one projection, the causal
convolution with SiLU over its channels, the delta rule (v a view of the convolution's
output), the gated RMS norm and the residual; trained through all of them, and a prompt
continued token by token from the state and the convolution's last inputs.

Against the same layer in float64.  The convolution's outputs are sums of four fp32
products, off by a few 2^-24 of their terms; the rest is as without it: 2^-14 of the root
mean square."""
import pytest

from test_delta_block_gpu import B, G, H, K, T, V, WIDTH, _built, close, inputs, operators, plain  # noqa: F401

pytestmark = pytest.mark.gpu
TAPS, CHANNELS = 4, 2 * G * K + H * V


def parameters():
    import torch
    gen = torch.Generator("cuda").manual_seed(13)
    r = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    return {"wn": 1 + r(WIDTH, std=0.1), "bn": r(WIDTH, std=0.1), "wp": r(WIDTH, CHANNELS, std=0.1),
            "wc": r(CHANNELS, TAPS, std=0.5), "bc": r(CHANNELS, std=0.1),
            "wa": r(WIDTH, H, std=0.1), "wb": r(WIDTH, H, std=0.1), "wz": r(WIDTH, H * V, std=0.1),
            "wg": 1 + r(H * V, std=0.1), "wo": r(H * V, WIDTH, std=0.1)}


def conv_of_library():
    import torch
    import state_space_model_analytic_gb300 as ssd

    class Conv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b, before):
            ctx.save_for_backward(x, w, b, before)
            return ssd.conv1d_silu_forward(x, w, b, before)

        @staticmethod
        def backward(ctx, dout):
            x, w, b, before = ctx.saved_tensors
            g = ssd.conv1d_silu_backward(x, w, b, before, dout.contiguous())
            return g["dx"], g["dweight"], g["dbias"], None
    return Conv.apply


def plain_conv(x, w, b, before):
    import torch
    line = torch.cat([before.transpose(1, 2).to(x.dtype), x], 1)
    n = x.shape[1]
    z = b + sum(w[:, i] * line[:, i + 1:i + 1 + n] for i in range(TAPS))
    return torch.nn.functional.silu(z)


def layer(x, before, s0, lens, p, conv, norm, delta, gated):
    """(output, state, the projection: what the convolution has read)"""
    import torch
    n = norm(x, p["wn"], p["bn"])
    u = (n @ p["wp"]).contiguous()
    c = conv(u, p["wc"], p["bc"], before)
    q, k, v = c.split([G * K, G * K, H * V], -1)
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    q, k, v = unit(q.unflatten(-1, (G, K))), unit(k.unflatten(-1, (G, K))), v.unflatten(-1, (H, V))
    la, be = -torch.nn.functional.softplus(n @ p["wa"] - 2), torch.sigmoid(n @ p["wb"])
    o, s = delta(q, k, v, la.contiguous(), be.contiguous(), s0, lens)
    return x + gated(o.flatten(-2), (n @ p["wz"]).contiguous(), p["wg"]) @ p["wo"], s, u


def history(seed=14):
    import torch
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(B, CHANNELS, TAPS, generator=gen, device="cuda")


@pytest.mark.parametrize("lens", [None, (90, 1, 64)])
def test_a_layer_and_its_gradients(lens):
    import torch
    x, s0 = inputs()
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(15)
    results = []
    for conv, ops, dt in ((conv_of_library(), operators(), torch.float32),
                          (plain_conv, plain(), torch.float64)):
        p = {n: t.to(dt).requires_grad_() for n, t in parameters().items()}
        xs, ss = x.to(dt).requires_grad_(), s0.to(dt).requires_grad_()
        y, s, _ = layer(xs, history(), ss, ln, p, conv, *ops)
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
    p, conv = parameters(), conv_of_library()
    norm, delta, gated = operators()
    y, s, _ = layer(x, history(), s0, None, p, conv, norm, delta, gated)
    y1, state, u = layer(x[:, :80].contiguous(), history(), s0, None, p, conv, norm, delta, gated)
    close(y1, y[:, :80].double())
    before = u[:, -TAPS:].transpose(1, 2).contiguous()

    def one(q, k, v, la, be, state, _):
        a = [t[:, 0].contiguous() for t in (q, k, v, la, be)]
        o, new = ssd.delta_rule_step(*a, state, scale=K ** -0.5)
        return o[:, None], new

    for t in range(80, 90):
        yt, state, u = layer(x[:, t:t + 1].contiguous(), before, state, None, p, conv, norm, one, gated)
        before = torch.cat([before[:, :, 1:], u.transpose(1, 2)], -1).contiguous()
        close(yt, y[:, t:t + 1].double())
    close(state, s.double())
