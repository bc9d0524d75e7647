"""Cases of the gated-delta-rule and layer-norm operators.

A delta-rule layer of a recurrent language model is normalised (layer norm),
mixed over time by a fast-weight memory that corrects what it holds for a key
before it writes (the gated delta rule) and trained through both; once trained
it reads prompts, continues them token by token and keeps one state a head.
The cases are those calls at the sizes of this repository's workloads and
around them.

    delta     e_t = v_t - a_t S_{t-1} k_t,  S_t = a_t S_{t-1} + beta_t e_t k_t^T,
              o_t = scale S_t q_t,  a_t = e^{log_decay_t}
              q, k [B, T, G, K], v [B, T, H, V] (head h uses group h / (H/G)),
              log_decay, beta [B, T, H], state [B, H, V, K]; rows may be shorter
              than T (lens)
    norm      y = (x - mean) / sqrt(var + eps) weight + bias over the last dimension
"""
import math

import torch

own = False

EPS_NORM = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def _delta(op, B, T, H, G, K, V, dtype, state, ragged, packed, name=None):
    c = {"op": op, "B": B, "T": T, "H": H, "G": G, "K": K, "V": V, "dtype": dtype,
         "state": state, "ragged": ragged, "packed": packed}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # prompts: the d_inner-2048 layer of the benchmark (32 heads of 64, state size 128), every
        # head with its own q and k, read as views of one buffer
        _delta("forward", 4, 2048, 32, 32, 128, 64, "bf16", False, False, True, "prompt_layer"),
        # one long document continued from a state: few rows, many steps
        _delta("forward", 1, 16384, 32, 4, 128, 64, "bf16", True, False, False, "prompt_long"),
        # a batch of prompts of different odd lengths, padded to the longest
        _delta("forward", 16, 1003, 24, 24, 64, 64, "bf16", True, True, False, "prompt_ragged"),
        # 32-bit activations: the fp32 workload's sizes
        _delta("forward", 8, 1024, 24, 24, 64, 64, "f32", True, False, False, "prompt_fp32"),
        # training: the gradients of the same layer, of heads that share q and k in groups and have
        # states of 128 x 128, and of a small 32-bit layer
        _delta("backward", 4, 2048, 32, 32, 128, 64, "bf16", False, False, False, "train_layer"),
        _delta("backward", 2, 4096, 32, 8, 128, 128, "bf16", True, False, False, "train_grouped"),
        _delta("backward", 2, 1000, 12, 12, 64, 64, "f32", True, True, False, "train_fp32"),
        # serving: one token of one stream (latency), and of a large batch (the states' bandwidth)
        _delta("step", 1, 1, 32, 32, 128, 64, "bf16", True, False, False, "token_single"),
        _delta("step", 256, 1, 64, 8, 128, 64, "bf16", True, False, False, "token_batch"),
        # before a block: a training batch of the benchmark (8192 tokens), forward and backward, and
        # the rows of a decoding batch in 32 bits at an odd width (latency)
        {"op": "norm_forward", "rows": 8192, "width": 2048, "dtype": "bf16", "bias": True,
         "name": "norm_layer"},
        {"op": "norm_backward", "rows": 8192, "width": 2048, "dtype": "bf16", "bias": True,
         "name": "norm_layer_grad"},
        {"op": "norm_forward", "rows": 250, "width": 1537, "dtype": "f32", "bias": True,
         "name": "norm_tokens"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "backward", "step",
                     "norm_forward", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        width = _log_int(rng, 64, 8192)
        # mostly odd multiples of a head's 64, else odd
        width = (width // 64 | 1) * 64 if rng.random() < 0.75 else width | 1
        width = min(width, 8191)
        return {"op": op, "rows": min(_log_int(rng, 1, 16384), (1 << 24) // width), "width": width,
                "dtype": dtype, "bias": rng.random() < 0.7}
    H = rng.choice([1, 2, 3, 8, 12, 24, 32, 64])
    G = rng.choice([g for g in (1, 2, 3, 4, 8, 12, 24, 32, 64) if H % g == 0] + [H, H])
    K = rng.choice([16, 32, 64, 64, 80, 128, 128])
    V = rng.choice([16, 32, 64, 64, 96, 128])
    if op == "step":
        return _delta(op, _log_int(rng, 1, 256), 1, H, G, K, V, dtype, True, False, False)
    # at most half of the largest case's tokens x heads (an eighth in 32 bits)
    most = (1 << 15) if dtype == "f32" else (1 << 17)
    T = _log_int(rng, 1, min(8192, most // H))
    B = _log_int(rng, 1, min(32, most // (T * H)))
    return _delta(op, B, T, H, G, K, V, dtype, rng.random() < 0.5, rng.random() < 0.4,
                  op == "forward" and rng.random() < 0.4)


# ---- inputs --------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    s = dict(case)
    io = TYPES[case["dtype"]]
    if case["op"].startswith("norm"):
        rows, width = case["rows"], case["width"]
        # a residual stream: columns of different size and offset
        s["x"] = (normal((rows, width)) * (0.5 + normal((width,)).abs()) + normal((width,), std=0.5)).to(io)
        s["weight"] = 1.0 + normal((width,), std=0.1)
        s["bias"] = normal((width,), std=0.1) if case["bias"] else None
        if case["op"] == "norm_backward":
            s["dy"] = normal((rows, width), io)
            # what the forward of the training step kept
            x = s["x"].double()
            mean = x.mean(-1)
            var = (x - mean[:, None]).square().mean(-1)
            s["stats"] = torch.stack([mean, (var + EPS_NORM).rsqrt()], -1).float()
        return s
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")

    def unit(shape):
        """What a short convolution with SiLU leaves, with rows of length 1."""
        x = normal(shape)
        x = x * torch.sigmoid(x)
        return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()

    q, k, v = unit((B, T, G, K)).to(io), unit((B, T, G, K)).to(io), normal((B, T, H, V), io)
    if case["packed"]:  # views of one buffer
        q, k, v = torch.cat([x.reshape(B, T, -1) for x in (q, k, v)], -1).split(
            [G * K, G * K, H * V], dim=-1)
        q, k, v = q.view(B, T, G, K), k.view(B, T, G, K), v.view(B, T, H, V)
    s["q"], s["k"], s["v"] = q, k, v
    s["scale"] = K ** -0.5
    # gates: time steps of 0.001 to 0.1 at rest, rates of 1 to 16 a head, write strengths in (0, 1)
    rate = 1.0 + 15.0 * torch.rand((H,), generator=gen, device=dev)
    rest = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((H,), generator=gen, device=dev))
    bias = rest + torch.log(-torch.expm1(-rest))
    s["log_decay"] = -rate * torch.nn.functional.softplus(normal((B, T, H)) + bias)
    s["beta"] = torch.sigmoid(normal((B, T, H)))
    s["state0"] = normal((B, H, V, K), std=0.5) if case["state"] else None
    s["lens"] = None
    if case["ragged"]:
        s["lens"] = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        s["lens"][B // 2] = T
    if case["op"] == "backward":
        s["do"] = normal((B, T, H, V), io)
        s["dstate"] = normal((B, H, V, K), std=0.1) if case["state"] else None
    if case["op"] == "step":
        for x in ("q", "k", "v", "log_decay", "beta"):
            s[x] = s[x][:, 0].contiguous()
        s["state_out"] = torch.empty_like(s["state0"])
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import state_space_model_analytic_gb300 as ssd
    op = s["op"]
    if op == "forward":
        o, state = ssd.delta_rule_forward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"],
                                          s["state0"], scale=s["scale"], lens=s["lens"])
        return {"o": o, "state": state}
    if op == "backward":
        return ssd.delta_rule_backward(s["q"], s["k"], s["v"], s["log_decay"], s["beta"],
                                       s["state0"], s["do"], s["dstate"], scale=s["scale"],
                                       lens=s["lens"])
    if op == "step":
        o, state = ssd.delta_rule_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"],
                                       s["state0"], scale=s["scale"], state_out=s["state_out"])
        return {"o": o, "state": state}
    if op == "norm_forward":
        y, _ = ssd.layer_norm_forward(s["x"], s["weight"], s["bias"], EPS_NORM, want_stats=False)
        return {"y": y}
    return ssd.layer_norm_backward(s["x"], s["weight"], s["dy"], EPS_NORM, s["stats"],
                                   want_dbias=s["bias"] is not None)


# ---- plain forms ---------------------------------------------------------------

CHUNK = 64


def _heads(x, H):
    """[B, T, G, D] -> [B, H, T, D] in 32 bits, each group's row for all of its heads."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _chunked(x, lens, T):
    """[B, H, T, ...] -> [B, H, chunks, CHUNK, ...], zero past each row's length."""
    if lens is not None:
        live = (torch.arange(T, device=x.device) < lens[:, None])[:, None, :]
        live = live.reshape(live.shape + (1,) * (x.dim() - 3))
        x = torch.where(live, x, torch.zeros((), device=x.device, dtype=x.dtype))
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[:2] + (pad,) + x.shape[3:])], 2)
    return x.reshape(x.shape[:2] + (n, CHUNK) + x.shape[3:])


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower triangular A [..., C, C], C a power of two: blocks of 1, 2,
    4 ... rows are joined, [[P, 0], [R, Q]]^-1 = [[P^-1, 0], [-Q^-1 R P^-1, Q^-1]]."""
    C = A.shape[-1]
    inv = torch.eye(C, device=A.device).expand(A.shape).clone()
    n = 1
    while n < C:
        def blocks(x, i, j):
            x = x.unflatten(-2, (C // (2 * n), 2, n)).unflatten(-1, (C // (2 * n), 2, n))
            return x[..., i, :, :, j, :].diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        low = blocks(inv, 1, 1) @ blocks(A, 1, 0) @ blocks(inv, 0, 0)
        at = inv.unflatten(-2, (C // (2 * n), 2, n)).unflatten(-1, (C // (2 * n), 2, n))
        at[..., 1, :, :, 0, :].diagonal(dim1=-4, dim2=-2).copy_(-low.movedim(-3, -1))
        n *= 2
    return inv


def _plain_chunks(s):
    """What every chunk holds, for all chunks at once."""
    T, H, lens = s["T"], s["H"], s["lens"]
    q, k, v = (_chunked(_heads(s[x], H), lens, T) for x in "qkv")
    beta = _chunked(s["beta"].transpose(1, 2), lens, T)[..., None]
    # sums of logarithms in 64 bits: their differences count
    g = _chunked(s["log_decay"].double().transpose(1, 2), lens, T).cumsum(-1)
    i = torch.arange(CHUNK, device=q.device)
    low = i[:, None] >= i[None, :]
    gamma = torch.where(low, torch.exp(torch.where(low, g[..., :, None] - g[..., None, :], 0.0).float()), 0.0)
    L = torch.where(i[:, None] > i[None, :], gamma * (k @ k.transpose(-1, -2)), 0.0)
    P = gamma * (q @ k.transpose(-1, -2))
    lead, tail = torch.exp(g.float())[..., None], torch.exp((g[..., -1:] - g).float())[..., None]
    return q, k, v, beta, gamma, L, P, _unit_lower_inverse(L * beta.transpose(-1, -2)), lead, tail


def _plain_walk(s, q, k, v, beta, inv, lead, tail):
    """The states before every chunk and after the last ([B, H, K, V]), and the errors e."""
    B, H, n = k.shape[:3]
    K, V = k.shape[-1], v.shape[-1]
    S = k.new_zeros(B, H, K, V) if s["state0"] is None else s["state0"].transpose(-1, -2)
    states, errors = [S], []
    read, write, last = lead * k, (tail * k).transpose(-1, -2), lead[..., -1:, :]
    for c in range(n):
        e = inv[:, :, c] @ (v[:, :, c] - read[:, :, c] @ S)
        S = last[:, :, c] * S + write[:, :, c] @ (beta[:, :, c] * e)
        states.append(S)
        errors.append(e)
    return torch.stack(states, 2), torch.stack(errors, 2)


def _plain_forward(s):
    B, T, H = s["B"], s["T"], s["H"]
    q, k, v, beta, _, _, P, inv, lead, tail = _plain_chunks(s)
    S, e = _plain_walk(s, q, k, v, beta, inv, lead, tail)
    o = s["scale"] * (lead * (q @ S[:, :, :-1]) + P @ (beta * e))
    o = o.reshape(B, H, -1, s["V"])[:, :, :T].transpose(1, 2)
    return {"o": o.to(s["q"].dtype).contiguous(), "state": S[:, :, -1].transpose(-1, -2).contiguous()}


def _plain_backward(s):
    B, T, H, G, K, V, lens = (s[x] for x in ("B", "T", "H", "G", "K", "V", "lens"))
    io = s["q"].dtype
    q, k, v, beta, gamma, L, P, inv, lead, tail = _plain_chunks(s)
    S, e = _plain_walk(s, q, k, v, beta, inv, lead, tail)
    do = _chunked(_heads(s["do"], H), lens, T) * s["scale"]
    u, n = beta * e, k.shape[2]
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    # back over the chunks: D = d/d state after the chunk, y = d/d e without beta's factor
    D = torch.zeros_like(S[:, :, 0]) if s["dstate"] is None else t(s["dstate"])
    du_local, d_local, inv_t = t(P) @ do, t(lead * q) @ do, t(inv)
    write, read, last = tail * k, t(lead * k), lead[..., -1:, :]
    Ds, dvs, ys = [None] * n, [None] * n, [None] * n
    for c in reversed(range(n)):
        Ds[c] = D
        du = du_local[:, :, c] + write[:, :, c] @ D
        # dv = d e = (I + L beta)^-T beta du; du - L^T dv is what reaches e through u
        dvs[c] = inv_t[:, :, c] @ (beta[:, :, c] * du)
        ys[c] = du - t(L[:, :, c]) @ dvs[c]
        D = last[:, :, c] * D + d_local[:, :, c] - read[:, :, c] @ dvs[c]
    dstate0 = t(D).contiguous()
    D, dv, y = (torch.stack(x, 2) for x in (Ds, dvs, ys))
    first, after = S[:, :, :-1], S[:, :, 1:]
    mp = gamma * (do @ t(u))                 # d (q k^T), with the decays
    i = torch.arange(CHUNK, device=q.device)
    ml = torch.where(i[:, None] > i[None, :], -gamma * (dv @ t(u)), 0.0)
    dq = lead * (do @ t(first)) + mp @ k
    dk_read = ml @ k - lead * (dv @ t(first))
    dk_write = t(mp) @ q + t(ml) @ k + tail * (u @ t(D))
    # decays: e^{g_i} goes with q_i and the reading k_i, e^{-g_i} with the writing k_i, and the
    # state after the chunk has e^{g_last}.  The terms cancel: in 64 bits
    dot = lambda a, b: (a.double() * b.double()).sum(-1)  # noqa: E731
    dg = dot(q, dq) + dot(k, dk_read) - dot(k, dk_write)
    dg[..., -1] += dot(after, D).sum(-1)
    dg = dg.flip(-1).cumsum(-1).flip(-1)
    rows = lambda x: x.reshape(B, H, n * CHUNK, -1)[:, :, :T]  # noqa: E731

    def finish(x, groups):
        x = rows(x)
        if lens is not None:
            live = (torch.arange(T, device=x.device) < lens[:, None])[:, None, :, None]
            x = torch.where(live, x, torch.zeros((), device=x.device, dtype=x.dtype))
        return x.reshape(B, groups, H // groups, T, -1).sum(2).transpose(1, 2)

    gate = lambda x: finish(x, H)[..., 0].float().contiguous()  # noqa: E731
    return {"dq": finish(dq, G).to(io).contiguous(),
            "dk": finish(dk_read + dk_write, G).to(io).contiguous(),
            "dv": finish(dv, H).to(io).contiguous(),
            "dlog_decay": gate(dg[..., None]), "dbeta": gate(dot(e, y)[..., None]),
            "dstate0": dstate0}


def _plain_step(s):
    r = s["H"] // s["G"]
    q, k = (s[x].float().repeat_interleave(r, dim=1)[:, :, None] for x in "qk")
    S = torch.exp(s["log_decay"])[..., None, None] * s["state0"]
    e = s["v"].float() - (S * k).sum(-1)
    S = S + (s["beta"][..., None] * e)[..., None] * k
    o = (S * q).sum(-1) * s["scale"]
    return {"o": o.to(s["q"].dtype), "state": S}


def _plain_norm_forward(s):
    x = s["x"].float()
    d = x - x.mean(-1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS_NORM) * s["weight"]
    return {"y": (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype)}


def _plain_norm_backward(s):
    dy, mean, inv = s["dy"].float(), s["stats"][:, :1], s["stats"][:, 1:]
    n = (s["x"].float() - mean) * inv
    t = dy * s["weight"]
    dx = inv * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0),
            "dbias": None if s["bias"] is None else dy.sum(0)}


_PLAIN = {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step,
          "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n, rows, width = case["rows"] * case["width"], case["rows"], case["width"]
        g = 1 if case["bias"] else 0
        if op == "norm_forward":
            return {"bytes": 2 * n * e + 4 * (1 + g) * width, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * rows + 4 * (2 + g) * width, "flops": 15 * n}
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")
    state = 4 * B * H * V * K
    if op == "step":
        return {"bytes": 2 * state + B * (2 * G * K + 2 * H * V) * e + 8 * B * H,
                "flops": 7 * B * H * V * K}
    # the recurrence itself: 3 products of V x K a step and head forward; backward 3 for the errors
    # and the states, 3 for the gradients of the states and 4 for those of q, k, v
    io = B * T * (2 * G * K + 2 * H * V) * e
    gates = 8 * B * T * H
    if op == "forward":
        return {"bytes": io + gates + state * (2 if case["state"] else 1),
                "flops": 6 * B * T * H * K * V}
    return {"bytes": 2 * io - B * T * H * V * e + 2 * gates + state * (3 if case["state"] else 1),
            "flops": 20 * B * T * H * K * V}


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(s)
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")
    S = torch.zeros(B, H, V, K, dtype=torch.float64, device="cuda") if s["state0"] is None \
        else s["state0"].double()
    spread = lambda x: x.double().repeat_interleave(H // G, dim=1)  # noqa: E731
    out = lambda M, x: torch.einsum("bhvk,bhk->bhv", M, x)  # noqa: E731

    def advance(S, k, v, la, beta):
        """(decayed state, error, state after the step)"""
        A = S * la.double().exp()[..., None, None]
        e = v.double() - out(A, k)
        return A, e, torch.addcmul(A, (beta.double()[..., None] * e)[..., None], k[:, :, None])

    if op == "step":
        S = advance(S, spread(s["k"]), s["v"], s["log_decay"], s["beta"])[2]
        return {"o": out(S, spread(s["q"])) * s["scale"], "state": S}
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    live = (torch.arange(T, device="cuda")[:, None] < lens)[:, :, None, None, None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    at = lambda t: (spread(s["k"][:, t]), s["v"][:, t], s["log_decay"][:, t], s["beta"][:, t])  # noqa: E731
    if op == "forward":
        o = torch.zeros(B, T, H, V, dtype=torch.float64, device="cuda")
        for t in range(T):  # the recurrence, step by step
            S = torch.where(live[t], advance(S, *at(t))[2], S)
            o[:, t] = torch.where(live[t][..., 0], out(S, spread(s["q"][:, t])) * s["scale"], zero)
        return {"o": o, "state": S}
    # gradients: the states of a stretch are computed again when its turn comes
    stretch = max(1, min(T, (1 << 27) // S.numel()))
    starts = []
    for t in range(T):
        if t % stretch == 0:
            starts.append(S)
        S = torch.where(live[t], advance(S, *at(t))[2], S)
    D = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    dq, dk = (torch.zeros(B, T, G, K, dtype=torch.float64, device="cuda") for _ in range(2))
    dv = torch.zeros(B, T, H, V, dtype=torch.float64, device="cuda")
    dg, db = (torch.zeros(B, T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    group = lambda x: x.reshape(B, G, H // G, K).sum(2)  # noqa: E731
    for first in reversed(range(0, T, stretch)):
        S, before = starts.pop(), []
        for t in range(first, min(T, first + stretch)):
            before.append(S)
            S = torch.where(live[t], advance(S, *at(t))[2], S)
        for t in reversed(range(first, min(T, first + stretch))):
            k, v, la, beta = at(t)
            A, e, S = advance(before.pop(), k, v, la, beta)
            beta, do = beta.double(), s["do"][:, t].double() * s["scale"]
            l3, l2 = live[t][..., 0], live[t][..., 0, 0]
            dq[:, t] = torch.where(l3, group(torch.einsum("bhvk,bhv->bhk", S, do)), zero)
            M = torch.addcmul(D, do[..., None], spread(s["q"][:, t])[:, :, None])  # d / d S_t
            Mk = out(M, k)
            db[:, t] = torch.where(l2, (e * Mk).sum(-1), zero)
            de = beta[..., None] * Mk
            dv[:, t] = torch.where(l3, de, zero)
            d = torch.einsum("bhvk,bhv->bhk", M, beta[..., None] * e) - torch.einsum("bhvk,bhv->bhk", A, de)
            dk[:, t] = torch.where(l3, group(d), zero)
            dA = M - de[..., None] * k[:, :, None]
            dg[:, t] = torch.where(l2, (dA * A).sum((-1, -2)), zero)
            D = torch.where(live[t], dA * la.double().exp()[..., None, None], D)
    return {"dq": dq, "dk": dk, "dv": dv, "dlog_decay": dg, "dbeta": db, "dstate0": D}


def _exact_norm(s):
    """The forward in 64 bits, and its gradients by torch's differentiation of it."""
    back = s["op"] == "norm_backward"
    x, w = (s[k].double().requires_grad_(back) for k in ("x", "weight"))
    b = None if s["bias"] is None else s["bias"].double().requires_grad_(back)
    var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
    y = (x - mean) / (var + EPS_NORM).sqrt() * w
    if b is not None:
        y = y + b
    if not back:
        return {"y": y}
    got = torch.autograd.grad(y, [x, w] + ([] if b is None else [b]), s["dy"].double())
    return {"dx": got[0], "dweight": got[1], "dbias": None if b is None else got[2]}
