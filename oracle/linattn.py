"""Float64 reference of linear attention with a decay for each head, step by
step from its definition (test infrastructure):

    S_t = a_h S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   a_h = exp(log_decay_h)

q, k [B,T,G,K], v, do [B,T,H,V]; head h reads group h // (H/G); row b has
lens[b] steps.  The backward is the adjoint of the recurrence,

    g_t = a g_{t+1} + scale do_t q_t^T  (g_n = dstate / a at the last step),
    dq_t = scale S_t^T do_t,  dk_t = g_t^T v_t,  dv_t = g_t k_t,  dS0 = a g_0.
"""
import numpy as np


def _spread(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def _live(lens, B, t):
    return np.array([t < (n if n is not None else t + 1) for n in (lens if lens is not None else [None] * B)])


def _decay(log_decay):
    return np.exp(np.asarray(log_decay, dtype=np.float64))[None, :, None, None]


def _clean(x, lens):
    """Zeros past each row's length (what lies there is not an input)."""
    x = np.array(x, dtype=np.float64)
    if lens is not None:
        for b, n in enumerate(lens):
            x[b, n:] = 0.0
    return x


def forward(q, k, v, log_decay, state0=None, scale=1.0, lens=None):
    """(o [B,T,H,V], state [B,H,V,K])"""
    q, k, v = (_clean(x, lens) for x in (q, k, v))
    B, T, H, V = v.shape
    K = q.shape[-1]
    a = _decay(log_decay)
    S = np.zeros((B, H, V, K)) if state0 is None else np.array(state0, dtype=np.float64)
    o = np.zeros((B, T, H, V))
    for t in range(T):
        live = _live(lens, B, t)[:, None, None, None]
        new = a * S + v[:, t, :, :, None] * _spread(k[:, t], H)[:, :, None, :]
        S = np.where(live, new, S)
        o[:, t] = np.where(live[..., 0], scale * np.einsum("bhvk,bhk->bhv", S, _spread(q[:, t], H)), 0)
    return o, S


def backward(q, k, v, log_decay, state0, do, dstate=None, scale=1.0, lens=None):
    """dict dq, dk [B,T,G,K], dv [B,T,H,V], dstate0 [B,H,V,K]"""
    q, k, v, do = (_clean(x, lens) for x in (q, k, v, do))
    B, T, H, V = v.shape
    G, K = q.shape[2], q.shape[3]
    a = _decay(log_decay)
    S = np.zeros((B, H, V, K)) if state0 is None else np.array(state0, dtype=np.float64)
    D = np.zeros((B, H, V, K)) if dstate is None else np.array(dstate, dtype=np.float64)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    group = lambda x: x.reshape(B, G, H // G, K).sum(2)  # noqa: E731
    for t in range(T):
        live = _live(lens, B, t)[:, None, None, None]
        S = np.where(live, a * S + v[:, t, :, :, None] * _spread(k[:, t], H)[:, :, None, :], S)
        y = scale * np.einsum("bhvk,bhv->bhk", S, do[:, t])
        dq[:, t] = np.where(live[..., 0], group(y), 0)
    for t in reversed(range(T)):
        live = _live(lens, B, t)[:, None, None, None]
        g = D + scale * do[:, t, :, :, None] * _spread(q[:, t], H)[:, :, None, :]
        dk[:, t] = np.where(live[..., 0], group(np.einsum("bhvk,bhv->bhk", g, v[:, t])), 0)
        dv[:, t] = np.where(live[..., 0], np.einsum("bhvk,bhk->bhv", g, _spread(k[:, t], H)), 0)
        D = np.where(live, a * g, D)
    return {"dq": dq, "dk": dk, "dv": dv, "dstate0": D}


def step(q, k, v, log_decay, state, scale=1.0):
    """One token: q, k [B,G,K], v [B,H,V], log_decay [H] or [B,H]; (o, state)."""
    H = v.shape[1]
    a = np.exp(np.broadcast_to(np.asarray(log_decay, dtype=np.float64), v.shape[:2]))[..., None, None]
    S = a * state + v[..., :, None] * _spread(k, H)[..., None, :]
    return scale * np.einsum("bhvk,bhk->bhv", S, _spread(q, H)), S
