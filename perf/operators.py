"""Cases of the linear-attention, block-norm and gradient-clipping operators.

One layer of a recurrent language model is normalised, mixed over time by
linear attention with a decay for each head, normalised again, gated and added
to the residual stream; its gradients are clipped by their global norm; once
trained it reads prompts and then continues them token by token.  The cases
are those calls at the sizes of this repository's workloads and around them.

    linattn   o_t = scale S_t q_t,  S_t = e^{log_decay_h} S_{t-1} + v_t k_t^T
              q, k [B, T, G, K], v [B, T, H, V] (head h uses group h / (H/G)),
              state [B, H, V, K]; rows may be shorter than T (lens)
    norm      r' = r + res_scale * (rmsnorm(y) w_post silu(z)),  x = rmsnorm(r') w_pre
    clip      n = sqrt(sum g^2) over all tensors,  g <- g min(1, max_norm / (n + 1e-6))
"""
import math

import torch

own = False

EPS_NORM = 1e-5
EPS_CLIP = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def _la(op, B, T, H, G, K, V, dtype, state, ragged, packed, name=None):
    c = {"op": op, "B": B, "T": T, "H": H, "G": G, "K": K, "V": V, "dtype": dtype,
         "state": state, "ragged": ragged, "packed": packed}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # prompts: the d_inner-2048 layer of the benchmark (32 heads of 64, state size 128), every
        # head with its own q and k, read as views of one projection's output
        _la("forward", 4, 2048, 32, 32, 128, 64, "bf16", False, False, True, "prompt_layer"),
        # one very long document continued from a state: the long-sequence workload's sizes
        _la("forward", 1, 32768, 32, 4, 128, 64, "bf16", True, False, False, "prompt_long"),
        # a batch of prompts of different odd lengths, padded to the longest
        _la("forward", 16, 1003, 24, 24, 64, 64, "bf16", True, True, False, "prompt_ragged"),
        # 32-bit activations: the fp32 workload's sizes
        _la("forward", 8, 1024, 24, 24, 64, 64, "f32", True, False, False, "prompt_fp32"),
        # training: the gradients of the same layer, and of heads that share q and k in groups
        # (the grouped workload), which are sums over a group's heads
        _la("backward", 4, 2048, 32, 32, 128, 64, "bf16", False, False, False, "train_layer"),
        _la("backward", 2, 8192, 64, 8, 128, 64, "bf16", True, False, False, "train_grouped"),
        # serving: one token of one stream (latency), and of a large batch (the states' bandwidth)
        _la("step", 1, 1, 32, 32, 128, 64, "bf16", True, False, False, "token_single"),
        _la("step", 256, 1, 64, 8, 128, 64, "bf16", True, False, False, "token_batch"),
        # between blocks, forward and backward, on a training batch of the benchmark (8192 tokens)
        {"op": "norm_forward", "rows": 8192, "width": 2048, "dtype": "bf16", "res": "f32",
         "gate": True, "name": "norm_layer"},
        {"op": "norm_backward", "rows": 8192, "width": 2048, "dtype": "bf16", "res": "f32",
         "gate": True, "name": "norm_layer_grad"},
        # a small model's gradients (latency), and a stack of layers (bandwidth)
        {"op": "clip", "tensors": 24, "largest": 147456, "dtype": "bf16", "max_norm": 1.0,
         "name": "clip_small"},
        {"op": "clip", "tensors": 240, "largest": 8388608, "dtype": "mixed", "max_norm": 1.0,
         "name": "clip_layers"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "step", "norm_forward",
                     "norm_backward", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        return {"op": op, "tensors": _log_int(rng, 1, 300), "largest": _log_int(rng, 1000, 4000000),
                "dtype": rng.choice(["bf16", "f32", "mixed"]),
                "max_norm": rng.choice([1.0, 0.5, 1e9])}
    if op.startswith("norm"):
        width = _log_int(rng, 64, 8192)
        # mostly odd multiples of a head's 64, else odd
        width = (width // 64 | 1) * 64 if rng.random() < 0.75 else width | 1
        return {"op": op, "rows": min(_log_int(rng, 1, 16384), (1 << 24) // width), "width": width,
                "dtype": dtype, "res": rng.choice(["f32", dtype]), "gate": rng.random() < 0.8}
    H = rng.choice([1, 2, 3, 8, 12, 24, 32, 64])
    G = rng.choice([g for g in (1, 2, 3, 4, 8, 12, 24, 32, 64) if H % g == 0] + [H, H])
    K = rng.choice([16, 32, 64, 64, 80, 128, 128])
    V = rng.choice([16, 32, 64, 64, 96, 128])
    if op == "step":
        return _la(op, _log_int(rng, 1, 256), 1, H, G, K, V, dtype, True, False, False)
    # at most half of the largest case's tokens x heads (an eighth in 32 bits)
    most = (1 << 17) if dtype == "f32" else (1 << 19)
    T = _log_int(rng, 1, min(16384, most // H))
    B = _log_int(rng, 1, min(32, most // (T * H)))
    return _la(op, B, T, H, G, K, V, dtype, rng.random() < 0.5, rng.random() < 0.4,
               op == "forward" and rng.random() < 0.4)


# ---- inputs --------------------------------------------------------------------

def _decays(H, dev):
    """Head h forgets over 32 to 512 steps: decays 1 - 2^-5 ... 1 - 2^-9."""
    e = torch.linspace(5.0, 9.0, H, device=dev) if H > 1 else torch.full((1,), 6.0, device=dev)
    return torch.log1p(-torch.exp2(-e))


def _clip_sizes(case):
    """Matrices of the largest size, halves of it and rows of weights, some odd."""
    L, row = case["largest"], max(1, int(math.sqrt(case["largest"])))
    return [(L, row, L // 2 + 1, row + 1, L // 4 + 3, 1)[i % 6] for i in range(case["tensors"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    s = dict(case)
    io = TYPES.get(case["dtype"])
    if case["op"] == "clip":
        sizes = _clip_sizes(case)
        kinds = [("bf16", "f32")[i % 2] if case["dtype"] == "mixed" else case["dtype"]
                 for i in range(len(sizes))]
        s["flat"], s["flat_out"], s["grads"], s["outs"] = {}, {}, [], []
        for kind in ("bf16", "f32"):
            mine = [n for n, k in zip(sizes, kinds) if k == kind]
            if mine:
                # gradients as a backward pass leaves them: one bucket a type
                s["flat"][kind] = normal((sum(mine),), TYPES[kind], 1e-3)
                s["flat_out"][kind] = torch.empty_like(s["flat"][kind])
                s["grads"] += list(s["flat"][kind].split(mine))
                s["outs"] += list(s["flat_out"][kind].split(mine))
        return s
    if case["op"].startswith("norm"):
        rows, width, res = case["rows"], case["width"], TYPES[case["res"]]
        s["y"] = normal((rows, width), io)
        s["z"] = normal((rows, width), io) if case["gate"] else None
        s["w_post"] = 1.0 + normal((width,), std=0.1)
        s["w_pre"] = 1.0 + normal((width,), std=0.1)
        s["res_scale"] = 0.2 + normal((width,), std=0.02)
        s["residual"] = normal((rows, width), res, 2.0)
        if case["op"] == "norm_backward":
            # the new residual and the gradients that reach it and the normed output
            s["dx"] = normal((rows, width), io)
            s["dres"] = normal((rows, width), res)
        return s
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")
    if case["packed"]:  # views of one projection's output
        qkv = normal((B, T, 2 * G * K + H * V), io)
        q, k, v = qkv.split([G * K, G * K, H * V], dim=-1)
        s["q"], s["k"], s["v"] = q.view(B, T, G, K), k.view(B, T, G, K), v.view(B, T, H, V)
    else:
        s["q"], s["k"] = normal((B, T, G, K), io), normal((B, T, G, K), io)
        s["v"] = normal((B, T, H, V), io)
    s["scale"] = K ** -0.5
    s["log_decay"] = _decays(H, dev)
    s["state0"] = normal((B, H, V, K)) if case["state"] else None
    s["lens"] = None
    if case["ragged"]:
        s["lens"] = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        s["lens"][B // 2] = T
    if case["op"] == "backward":
        s["do"] = normal((B, T, H, V), io)
        s["dstate"] = normal((B, H, V, K)) if case["state"] else None
    if case["op"] == "step":
        s["q"], s["k"], s["v"] = s["q"][:, 0], s["k"][:, 0], s["v"][:, 0]
        s["state_out"] = torch.empty_like(s["state0"])
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import state_space_model_analytic_gb300 as ssd
    op = s["op"]
    if op == "forward":
        o, state = ssd.linattn_forward(s["q"], s["k"], s["v"], s["log_decay"], s["state0"],
                                       scale=s["scale"], lens=s["lens"])
        return {"o": o, "state": state}
    if op == "backward":
        return ssd.linattn_backward(s["q"], s["k"], s["v"], s["log_decay"], s["state0"], s["do"],
                                    s["dstate"], scale=s["scale"], lens=s["lens"])
    if op == "step":
        o, state = ssd.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state0"],
                                    scale=s["scale"], state_out=s["state_out"])
        return {"o": o, "state": state}
    if op == "norm_forward":
        r, x, _ = ssd.block_norm_forward(s["residual"], s["y"], s["z"], s["w_post"],
                                         s["res_scale"], s["w_pre"], EPS_NORM, want_stats=False)
        return {"residual": r, "x": x}
    if op == "norm_backward":
        return ssd.block_norm_backward(s["residual"], s["y"], s["z"], s["w_post"],
                                       s["res_scale"], s["w_pre"], EPS_NORM, s["dx"], s["dres"])
    norm = ssd.clip_grad_norm(s["grads"], s["max_norm"], eps=EPS_CLIP, out=s["outs"])
    return {"norm": norm, "grads": s["flat_out"]}


# ---- plain forms ---------------------------------------------------------------

def _heads(x, H):
    """[B, T, G, D] -> [B, H, T, D] in 32 bits, each group's row for all of its heads."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _masked(x, lens, T):
    """Zero past each row's length (x [B, H, T, D])."""
    if lens is None:
        return x
    valid = torch.arange(T, device=x.device) < lens[:, None]
    return torch.where(valid[:, None, :, None], x, torch.zeros((), device=x.device))


def _walk(q, k, v, log_a, first, off, C=128):
    """sum_{j <= i} a^{i-j} (q_i . k_j) v_j + a^{i+off} first q_i, by chunks of C
    ([B, H, T, D] in 32 bits; first [B, H, Dv, Dk])."""
    B, H, T, Dk = q.shape
    Dv = v.shape[-1]
    C = min(C, T)
    n = -(-T // C)
    pad = n * C - T
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
    q, k, v = (x.reshape(B, H, n, C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    c = torch.arange(n, device=q.device, dtype=torch.float32)
    la = log_a[:, None, None]
    d = i[:, None] - i[None, :]
    inside = torch.where(d >= 0, torch.exp(la * d.clamp(min=0)), 0.0)           # [H, C, C]
    o = ((q @ k.transpose(-1, -2)) * inside[None, :, None]) @ v
    tail = torch.exp(log_a[:, None] * (C - 1 - i))[None, :, None, :, None]
    local = (v * tail).transpose(-1, -2) @ k                                    # [B,H,n,Dv,Dk]
    gap = c[:, None] - c[None, :] - 1
    across = torch.where(gap >= 0, torch.exp(la * C * gap.clamp(min=0)), 0.0)   # [H, n, n]
    before = (across[None] @ local.reshape(B, H, n, Dv * Dk)).reshape(B, H, n, Dv, Dk)
    lead = torch.exp(log_a[:, None] * (i + 1))[None, :, None, :, None]
    o = o + lead * (q @ before.transpose(-1, -2))
    if first is not None:
        t = i[None, :] + C * c[:, None] + off
        w = torch.exp(log_a[:, None, None] * t)[None, ..., None]
        o = o + w * (q @ first[:, :, None].transpose(-1, -2))
    return o.reshape(B, H, n * C, Dv)[:, :, :T]


def _flip(x, lens, T):
    """Reverses the first lens[b] steps of each row (x [B, H, T, D])."""
    if lens is None:
        return x.flip(2)
    t = torch.arange(T, device=x.device)
    at = torch.where(t < lens[:, None], lens[:, None] - 1 - t, t).long()
    return x.gather(2, at[:, None, :, None].expand(x.shape))


def _powers(log_a, lens, B, T, shift):
    """a^{len - 1 - t + shift} for t < len, 0 past it: [B, H, T]."""
    t = torch.arange(T, device=log_a.device, dtype=torch.float32)
    n = (lens.float() if lens is not None else torch.full((B,), float(T), device=log_a.device))
    e = n[:, None] - 1 - t + shift
    w = torch.exp(log_a[None, :, None] * e.clamp(min=0)[:, None, :])
    return torch.where((t < n[:, None])[:, None, :], w, 0.0), n


def _plain_forward(s):
    B, T, H, lens, log_a = s["B"], s["T"], s["H"], s["lens"], s["log_decay"]
    q, k, v = (_masked(_heads(s[x], H), lens, T) for x in "qkv")
    o = _walk(q, k, v, log_a, s["state0"], 1.0) * s["scale"]
    w, n = _powers(log_a, lens, B, T, 0.0)
    state = (v * w[..., None]).transpose(-1, -2) @ k
    if s["state0"] is not None:
        state = state + torch.exp(log_a[None] * n[:, None])[..., None, None] * s["state0"]
    return {"o": o.transpose(1, 2).to(s["q"].dtype).contiguous(), "state": state}


def _plain_backward(s):
    B, T, H, G, lens, log_a = s["B"], s["T"], s["H"], s["G"], s["lens"], s["log_decay"]
    io = s["q"].dtype
    q, k, v, do = (_masked(_heads(s[x], H), lens, T) for x in ("q", "k", "v", "do"))
    do = do * s["scale"]
    first = None if s["state0"] is None else s["state0"].transpose(-1, -2)
    dq = _walk(do, v, k, log_a, first, 1.0)
    fq, fk, fv, fdo = (_flip(x, lens, T) for x in (q, k, v, do))
    last = s["dstate"]
    dk = _flip(_walk(fv, fdo, fq, log_a, None if last is None else last.transpose(-1, -2), 0.0), lens, T)
    dv = _flip(_walk(fk, fq, fdo, log_a, last, 0.0), lens, T)
    dq, dk, dv = (_masked(x, lens, T) for x in (dq, dk, dv))
    t = torch.arange(T, device=q.device, dtype=torch.float32)
    w = torch.exp(log_a[:, None] * (t + 1))
    dstate0 = (do * w[None, ..., None]).transpose(-1, -2) @ q
    if last is not None:
        n = lens.float() if lens is not None else torch.full((B,), float(T), device=q.device)
        dstate0 = dstate0 + torch.exp(log_a[None] * n[:, None])[..., None, None] * last
    group = lambda x: x.reshape(B, G, H // G, T, -1).sum(2).transpose(1, 2).to(io).contiguous()  # noqa: E731
    return {"dq": group(dq), "dk": group(dk), "dv": dv.transpose(1, 2).to(io).contiguous(),
            "dstate0": dstate0}


def _plain_step(s):
    r = s["H"] // s["G"]
    q, k = (s[x].float().repeat_interleave(r, dim=1) for x in "qk")
    v = s["v"].float()
    state = (torch.exp(s["log_decay"])[None, :, None, None] * s["state0"] +
             v[..., :, None] * k[..., None, :])
    o = (state * q[..., None, :]).sum(-1) * s["scale"]
    return {"o": o.to(s["q"].dtype), "state": state}


def _plain_norm_forward(s):
    y, r = s["y"].float(), s["residual"].float()
    u = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS_NORM) * s["w_post"]
    if s["z"] is not None:
        z = s["z"].float()
        u = u * (z / (1.0 + torch.exp(-z)))
    new = r + s["res_scale"] * u
    x = new * torch.rsqrt(new.square().mean(-1, keepdim=True) + EPS_NORM) * s["w_pre"]
    return {"residual": new.to(s["residual"].dtype), "x": x.to(s["y"].dtype)}


def _plain_norm_backward(s):
    # `residual` is the forward's new residual here
    io, width = s["y"].dtype, s["y"].shape[-1]
    y, r, dx = s["y"].float(), s["residual"].float(), s["dx"].float()
    inv_r = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS_NORM)
    t = dx * s["w_pre"]
    dr = s["dres"].float() + inv_r * (t - r * inv_r * inv_r * ((t * r).sum(-1, keepdim=True) / width))
    inv_y = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS_NORM)
    normed = y * inv_y
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        gate, slope = z * sig, sig * (1.0 + z * (1.0 - sig))
    else:
        gate, slope = torch.ones((), device=y.device), None
    du = s["res_scale"] * dr
    dn = du * gate * s["w_post"]
    out = {"dresidual": dr.to(s["residual"].dtype),
           "dy": (inv_y * (dn - normed * inv_y * ((dn * y).sum(-1, keepdim=True) / width))).to(io),
           "dz": None if slope is None else (du * normed * s["w_post"] * slope).to(io),
           "dw_post": (du * gate * normed).sum(0),
           "dres_scale": (dr * normed * s["w_post"] * gate).sum(0),
           "dw_pre": (dx * r * inv_r).sum(0)}
    return out


def _plain_clip(s):
    flats = s["flat"]
    norm = torch.sqrt(torch.stack([f.float().square().sum() for f in flats.values()]).sum())
    coef = torch.clamp(s["max_norm"] / (norm + EPS_CLIP), max=1.0)
    return {"norm": norm, "grads": {k: (f.float() * coef).to(f.dtype) for k, f in flats.items()}}


_PLAIN = {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step,
          "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward,
          "clip": _plain_clip}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _clip_sizes(case)
        each = [{"bf16": 2, "f32": 4, "mixed": (2, 4)[i % 2]}[case["dtype"]] for i in range(len(sizes))]
        return {"bytes": 2 * sum(n * e for n, e in zip(sizes, each)), "flops": 3 * sum(sizes)}
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n, er = case["rows"] * case["width"], 2 if case["res"] == "bf16" else 4
        g = 1 if case["gate"] else 0
        if op == "norm_forward":
            return {"bytes": n * (2 * er + (2 + g) * e) + 12 * case["width"], "flops": (14 + 6 * g) * n}
        return {"bytes": n * (3 * er + (3 + 2 * g) * e) + 24 * case["width"], "flops": (30 + 12 * g) * n}
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")
    state = 4 * B * H * V * K
    if op == "step":
        return {"bytes": 2 * state + B * (2 * G * K + 2 * H * V) * e, "flops": 5 * B * H * V * K}
    # the recurrence itself: 2 products of V x K a step and head forward, 5 backward
    io = B * T * (2 * G * K + 2 * H * V) * e
    if op == "forward":
        return {"bytes": io + state * (2 if case["state"] else 1), "flops": 4 * B * T * H * K * V}
    return {"bytes": 2 * io - B * T * H * V * e + state * (3 if case["state"] else 1),
            "flops": 10 * B * T * H * K * V}


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            total += torch.dot(g.double(), g.double())
        norm = total.sqrt()
        coef = min(1.0, case["max_norm"] / (norm.item() + EPS_CLIP))
        return {"norm": norm, "grads": {k: f.double() * coef for k, f in s["flat"].items()}}
    if op.startswith("norm"):
        return _exact_norm(s)
    B, T, H, G, K, V = (case[k] for k in "BTHGKV")
    a = s["log_decay"].double().exp()[None, :, None, None]
    S = torch.zeros(B, H, V, K, dtype=torch.float64, device="cuda") if s["state0"] is None \
        else s["state0"].double()
    spread = lambda x: x.double().repeat_interleave(H // G, dim=1)  # noqa: E731
    if op == "step":
        S = a * S + s["v"].double()[..., None] * spread(s["k"])[:, :, None]
        o = (S @ spread(s["q"])[..., None])[..., 0] * case["K"] ** -0.5
        return {"o": o, "state": S}
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    live = torch.tensor([[t < n for n in lens] for t in range(T)], device="cuda")[:, :, None, None, None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    o = torch.zeros(B, T, H, V, dtype=torch.float64, device="cuda") if op == "forward" else None
    dq = torch.zeros(B, T, G, K, dtype=torch.float64, device="cuda") if op == "backward" else None
    for t in range(T):  # the recurrence, step by step
        kt, vt = spread(s["k"][:, t]), s["v"][:, t].double()
        S = torch.where(live[t], a * S + vt[..., None] * kt[:, :, None], S)
        if op == "forward":
            y = (S @ spread(s["q"][:, t])[..., None])[..., 0] * s["scale"]
            o[:, t] = torch.where(live[t][..., 0], y, zero)
        else:
            y = (s["do"][:, t].double()[:, :, None] @ S)[:, :, 0] * s["scale"]
            y = y.reshape(B, G, H // G, K).sum(2)
            dq[:, t] = torch.where(live[t][..., 0], y, zero)
    if op == "forward":
        return {"o": o, "state": S}
    dk, dv = torch.zeros_like(dq), torch.zeros(B, T, H, V, dtype=torch.float64, device="cuda")
    D = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()  # d / d S_t, later steps
    for t in reversed(range(T)):
        g = D + s["scale"] * s["do"][:, t].double()[..., None] * spread(s["q"][:, t])[:, :, None]
        y = (s["v"][:, t].double()[:, :, None] @ g)[:, :, 0].reshape(B, G, H // G, K).sum(2)
        dk[:, t] = torch.where(live[t][..., 0], y, zero)
        y = (g @ spread(s["k"][:, t])[..., None])[..., 0]
        dv[:, t] = torch.where(live[t][..., 0], y, zero)
        D = torch.where(live[t], a * g, D)
    return {"dq": dq, "dk": dk, "dv": dv, "dstate0": D}


def _exact_norm(s):
    """The forward in 64 bits, and its gradients by torch's differentiation of it."""
    back = s["op"] == "norm_backward"
    y = s["y"].double().requires_grad_(back)
    z = None if s["z"] is None else s["z"].double().requires_grad_(back)
    wp, wq, al = (s[k].double().requires_grad_(back) for k in ("w_post", "w_pre", "res_scale"))
    new = s["residual"].double()
    u = y / (y.pow(2).mean(-1, keepdim=True) + EPS_NORM).sqrt() * wp
    if z is not None:
        u = u * z * torch.sigmoid(z)
    add = al * u
    r = (new if back else new + add).detach().requires_grad_(back)
    x = r / (r.pow(2).mean(-1, keepdim=True) + EPS_NORM).sqrt() * wq
    if not back:
        return {"residual": r, "x": x}
    dr, dwq = torch.autograd.grad(x, [r, wq], s["dx"].double())
    dr = dr + s["dres"].double()
    ins = [y, wp, al] + ([] if z is None else [z])
    got = torch.autograd.grad(add, ins, dr)
    return {"dresidual": dr, "dy": got[0], "dz": None if z is None else got[3],
            "dw_post": got[1], "dres_scale": got[2], "dw_pre": dwq}
