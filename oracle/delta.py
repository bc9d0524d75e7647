"""Float64 reference of the gated delta rule, step by step from its definition
(test infrastructure):

    A_t = a_t S_{t-1},  e_t = v_t - A_t k_t,  S_t = A_t + beta_t e_t k_t^T,
    o_t = scale S_t q_t,  a_t = exp(log_decay_t)

q, k [B,T,G,K], v, do [B,T,H,V], log_decay, beta [B,T,H]; head h reads group
h // (H/G); row b has lens[b] steps.  The backward is the adjoint of the
recurrence: with M_t the gradient of S_t,

    M_t = D_t + scale do_t q_t^T,  D_t = a_{t+1} (M_{t+1} - de_{t+1} k_{t+1}^T),
    de_t = beta_t M_t k_t = dv_t,  dbeta_t = e_t . M_t k_t,
    dk_t = M_t^T beta_t e_t - A_t^T de_t,  dlog_decay_t = <M_t - de_t k_t^T, A_t>

Beside the values, the sizes that rounding errors go by: products of the norms of
what is multiplied (Cauchy and Schwarz), with the largest norm that a state has had,
decayed since (1 - beta k k^T does not lengthen it while beta |k|^2 <= 2), and the
largest of 64 steps to either side, whose terms a chunk adds up together.
"""
import numpy as np

WINDOW = 64


def _spread(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def _clean(x, lens):
    """Zeros past each row's length (what lies there is not an input)."""
    x = np.array(x, dtype=np.float64)
    if lens is not None:
        for b, n in enumerate(lens):
            x[b, n:] = 0.0
    return x


def _live(lens, B, T):
    n = np.full(B, T) if lens is None else np.asarray(lens)
    return np.arange(T)[:, None] < n  # [T, B]


def _norm(x, axes):
    return np.sqrt((x * x).sum(axes))


def _near(x):
    """The largest over WINDOW steps to either side (axis 1)."""
    T = x.shape[1]
    out = x.copy()
    for t in range(T):
        out[:, t] = x[:, max(0, t - WINDOW):t + WINDOW + 1].max(1)
    return out


def _advance(S, k, v, la, beta):
    A = np.exp(la)[..., None, None] * S
    e = v - np.einsum("bhvk,bhk->bhv", A, k)
    return A, e, A + (beta[..., None] * e)[..., None] * k[:, :, None]


def forward(q, k, v, log_decay, beta, state0=None, scale=1.0, lens=None):
    """(o [B,T,H,V], state [B,H,V,K], sizes of o, of the state's rows [B,H,V,1])"""
    q, k, v, log_decay, beta = (_clean(x, lens) for x in (q, k, v, log_decay, beta))
    B, T, H, V = v.shape
    S = np.zeros((B, H, V, q.shape[-1])) if state0 is None else np.array(state0, dtype=np.float64)
    o, size = np.zeros((B, T, H, V)), np.zeros((B, T, H, V))
    row, writes = _norm(S, -1), np.zeros((B, H, V))
    live = _live(lens, B, T)
    for t in range(T):
        on = live[t][:, None, None, None]
        kt, qt = _spread(k[:, t], H), _spread(q[:, t], H)
        A, e, new = _advance(S, kt, v[:, t], log_decay[:, t], beta[:, t])
        S = np.where(on, new, S)
        a, nk = np.exp(log_decay[:, t])[..., None], _norm(kt, -1)[..., None]
        w = np.abs(beta[:, t])[..., None] * (np.abs(v[:, t]) + _norm(A, -1) * nk) * nk
        row = np.where(on[..., 0], np.maximum.reduce([a * row, _norm(S, -1), w]), row)
        writes = np.where(on[..., 0], a * writes + w, writes)
        o[:, t] = np.where(on[..., 0], scale * np.einsum("bhvk,bhk->bhv", S, qt), 0)
        size[:, t] = abs(scale) * _norm(qt, -1)[..., None] * (row + writes)
    return o, S, _near(size), row[..., None]


def backward(q, k, v, log_decay, beta, state0, do, dstate=None, scale=1.0, lens=None):
    """(dict dq, dk, dv, dlog_decay, dbeta, dstate0; dict of their sizes)"""
    q, k, v, do, log_decay, beta = (_clean(x, lens) for x in (q, k, v, do, log_decay, beta))
    B, T, H, V = v.shape
    G, K = q.shape[2], q.shape[3]
    S = np.zeros((B, H, V, K)) if state0 is None else np.array(state0, dtype=np.float64)
    D = np.zeros((B, H, V, K)) if dstate is None else np.array(dstate, dtype=np.float64)
    live = _live(lens, B, T)
    kept, nS = [], np.zeros((B, T, H))
    run = _norm(S, (-1, -2))
    for t in range(T):
        on = live[t][:, None, None, None]
        A, e, new = _advance(S, _spread(k[:, t], H), v[:, t], log_decay[:, t], beta[:, t])
        S = np.where(on, new, S)
        kept.append((A, e, S))
        nk = _norm(_spread(k[:, t], H), -1)
        w = np.abs(beta[:, t]) * (_norm(v[:, t], -1) + run * nk) * nk
        run = np.maximum.reduce([np.exp(log_decay[:, t]) * run, _norm(S, (-1, -2)), w])
        nS[:, t] = run
    group = lambda x: x.reshape(B, G, H // G, -1).sum(2)  # noqa: E731
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v),
         "dlog_decay": np.zeros((B, T, H)), "dbeta": np.zeros((B, T, H))}
    size = {n: np.zeros((B, T, H)) for n in g}
    run = _norm(D, (-1, -2))
    for t in reversed(range(T)):
        on = live[t][:, None, None, None]
        A, e, St = kept[t]
        kt, qt, b = _spread(k[:, t], H), _spread(q[:, t], H), beta[:, t]
        dot = scale * do[:, t]
        M = D + dot[..., None] * qt[:, :, None]
        Mk = np.einsum("bhvk,bhk->bhv", M, kt)
        de = b[..., None] * Mk
        dA = M - de[..., None] * kt[:, :, None]
        g["dq"][:, t] = np.where(on[..., 0], group(np.einsum("bhvk,bhv->bhk", St, dot)), 0)
        g["dk"][:, t] = np.where(on[..., 0], group(
            np.einsum("bhvk,bhv->bhk", M, b[..., None] * e) - np.einsum("bhvk,bhv->bhk", A, de)), 0)
        g["dv"][:, t] = np.where(on[..., 0], de, 0)
        g["dbeta"][:, t] = np.where(on[..., 0, 0], (e * Mk).sum(-1), 0)
        g["dlog_decay"][:, t] = np.where(on[..., 0, 0], (dA * A).sum((-1, -2)), 0)
        nk, nq, ndo = _norm(kt, -1), _norm(qt, -1), _norm(dot, -1)
        run = np.where(on[..., 0, 0], np.maximum(run, ndo * nq), run)  # of M
        s, b = nS[:, t], np.abs(b)
        ne = _norm(v[:, t], -1) + s * nk
        for name, x in (("dq", s * ndo), ("dk", run * b * ne + s * b * run * nk), ("dv", b * run * nk),
                        ("dbeta", ne * run * nk), ("dlog_decay", s * run)):
            size[name][:, t] = x
        D = np.where(on, np.exp(log_decay[:, t])[..., None, None] * dA, D)
        run = np.where(on[..., 0, 0], np.maximum(np.exp(log_decay[:, t]) * run,
                                                 _norm(D, (-1, -2))), run)
    g["dstate0"] = D
    size = {n: _near(x) for n, x in size.items()}
    for n in ("dq", "dk"):
        size[n] = size[n].reshape(B, T, G, H // G).sum(-1)[..., None]
    size["dv"] = size["dv"][..., None]
    size["dstate0"] = run[..., None, None]
    return g, size


def step(q, k, v, log_decay, beta, state, scale=1.0):
    """One token: q, k [B,G,K], v [B,H,V], log_decay, beta [B,H]; (o, state)."""
    H = v.shape[1]
    S = _advance(np.asarray(state, dtype=np.float64), _spread(k, H), v, log_decay, beta)[2]
    return scale * np.einsum("bhvk,bhk->bhv", S, _spread(q, H)), S
