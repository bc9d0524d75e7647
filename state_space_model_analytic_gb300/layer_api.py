"""Python front end of the layer operators: linear attention with a decay for
each head, norms around a block, gradient clipping.  Torch CUDA tensors in, torch
tensors out; every step runs in the library's kernels behind the C ABI
(include/ssd.h), on `stream` or the current stream of the current device, whose
tensors they have to be.  A call on another stream
than the current one starts after the work that is on the current one, and its
operands may be dropped as soon as it returns.
"""
from __future__ import annotations

import array
import operator

import torch

from . import _native as nat
from . import _streams
from ._streams import check_device as _check_device

_IO_TYPES = {torch.float32: nat.SSD_F32, torch.bfloat16: nat.SSD_BF16}


_entry = {}


def _call(name):
    """The library's entry point, looked up once."""
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(nat.lib(), name)
    return f


def _ptr(t):
    return None if t is None else t.data_ptr()


def _size(t):
    return 0 if t is None else t.numel() * t.element_size()


class _Layouts(dict):
    """What a call derives from its operands' shapes, strides and types alone
    (never from their addresses or values), kept for the next call with the
    same ones."""

    def keep(self, key, value):
        if len(self) >= 1024:
            self.clear()
        self[key] = value
        return value


_layouts = _Layouts()


def _expect(name, t, dtype, shape, device, dense=True):
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _workspace(workspace, need, dev):
    """The caller's workspace after its checks (its size is the library's), or
    `need` bytes."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev:
        raise ValueError(f"workspace: on {workspace.device}, expected {dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace


def _io_type(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (no CPU path exists)")
    code = _IO_TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


# ---- linear attention ------------------------------------------------------------

def _rows_dense(name, t):
    """The last two dimensions are dense: the others are passed as strides."""
    if t.stride(-1) != 1 or (t.shape[-2] > 1 and t.stride(-2) != t.shape[-1]):
        raise ValueError(f"{name}: the last two dimensions must be contiguous")


def _linattn_dims(q, k, v, scale, log_decay, do, step):
    """(dims, workspace bytes forward, backward) after the operands' checks."""
    scale = float(scale)
    key = (step, q.shape, q.stride(), q.dtype, k.shape, k.stride(), k.dtype, v.shape, v.stride(),
           v.dtype, log_decay.shape, log_decay.dtype, log_decay.is_contiguous(), scale,
           None if do is None else (do.shape, do.stride(), do.dtype))
    dev = q.device
    if not q.is_cuda:
        raise ValueError("q: must be a CUDA tensor (no CPU path exists)")
    for name, t in (("k", k), ("v", v), ("log_decay", log_decay), ("do", do)):
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, expected {dev}")
    got = _layouts.get(key)
    if got is not None:
        return got
    code = _io_type("q", q)
    if q.dim() != (3 if step else 4):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected "
                         + ("[B, G, K]" if step else "[B, T, G, K]"))
    if v.dim() != q.dim():
        raise ValueError(f"v: {v.dim()} dimensions, expected {q.dim()}")
    B, G, K = q.shape[0], q.shape[-2], q.shape[-1]
    T = 1 if step else q.shape[1]
    H, V = v.shape[-2], v.shape[-1]
    _expect("k", k, q.dtype, q.shape, dev, False)
    _expect("v", v, q.dtype, (*q.shape[:-2], H, V), dev, False)
    if do is not None:
        _expect("do", do, v.dtype, v.shape, dev, False)
    for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
        if t is not None:
            _rows_dense(name, t)
    _expect("log_decay", log_decay, torch.float32,
            (B, H) if step and log_decay.dim() == 2 else (H,), dev)
    s = (lambda t: (t.stride(0), 0)) if step else (lambda t: (t.stride(0), t.stride(1)))
    d = nat.LinattnDims(B, T, H, G, K, V, *s(q), *s(k), *s(v), *(s(do) if do is not None else (0, 0)),
                        scale, code)
    size = _call("ssd_linattn_workspace_bytes")
    need = size(d, 0), size(d, 1)
    if not all(need):
        raise nat.SsdError(nat.SSD_ERR_UNSUPPORTED, nat.last_error() or "dims rejected")
    return _layouts.keep(key, (d, *need))


def _linattn_checks(d, dev, states, lens):
    shape = (d.batch, d.nheads, d.dv, d.dk)
    for name, t in states:
        if t is not None:
            _expect(name, t, torch.float32, shape, dev)
    if lens is not None:
        _expect("lens", lens, torch.int32, (d.batch,), dev)
    return shape


def linattn_workspace_bytes(q, k, v, log_decay, *, backward=False) -> int:
    """Bytes of the `workspace` that linattn_forward (or _backward) takes."""
    return _linattn_dims(q, k, v, 1.0, log_decay, None, False)[2 if backward else 1]


def linattn_forward(q, k, v, log_decay, state0=None, *, scale=1.0, lens=None, want_state=True,
                    out=None, workspace=None, stream=None):
    """Linear attention with a decay for each head over [B, T] steps:
    S_t = exp(log_decay_h) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.

    q, k [B,T,G,K], v [B,T,H,V] (fp32 or bf16; head h uses group h // (H/G);
    the last two dimensions contiguous, the others may be strided); log_decay
    [H] fp32, <= 0; state0 [B,H,V,K] fp32 or None (zeros); lens [B] int32 on
    the device: row b has lens[b] steps (o is zero past them).  K and V are
    multiples of 8 up to 128.  Returns (o [B,T,H,V], final state [B,H,V,K] or
    None); out: dict of preallocated "o", "state".

    State and sums are fp32.  bf16 operands: the decayed scores, and the state
    where it is multiplied, are rounded to bf16 once (o is off by 0.0023 of its
    root mean square, 0.0017 of which is its own rounding)."""
    d, need, _ = _linattn_dims(q, k, v, scale, log_decay, None, False)
    dev = q.device
    _check_device(dev, stream)
    out = {} if out is None else out
    o, state = out.get("o"), out.get("state")
    shape = _linattn_checks(d, dev, (("state0", state0), ("out state", state)), lens)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=dev)
    else:
        _expect("out o", o, v.dtype, v.shape, dev)
    if state is None and want_state:
        state = torch.empty(shape, dtype=torch.float32, device=dev)
    if workspace is not None or need > 256:
        workspace = _workspace(workspace, need, dev)
    _streams.keep(stream, q, k, v, log_decay, state0, lens, o, state, workspace)
    nat.check(_call("ssd_linattn_forward")(
        d, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(state0),
        _ptr(lens), o.data_ptr(), _ptr(state), _ptr(workspace), _size(workspace),
        _streams.handle(stream, dev)))
    return o, state


def linattn_backward(q, k, v, log_decay, state0, do, dstate=None, *, scale=1.0, lens=None,
                     want_dstate0=True, out=None, workspace=None, stream=None):
    """Gradients of sum(do * o) + sum(dstate * state) of linattn_forward: dict
    dq, dk, dv, dstate0 (or None).  do [B,T,H,V] may be strided like v;
    dstate [B,H,V,K] fp32 or None (zero).  log_decay gets no gradient.  Rounded
    as the forward's; in bf16 dq and dk come from states rounded to bf16."""
    d, _, need = _linattn_dims(q, k, v, scale, log_decay, do, False)
    dev = q.device
    _check_device(dev, stream)
    g = dict(out) if out is not None else {}
    shape = _linattn_checks(d, dev, (("state0", state0), ("dstate", dstate),
                                     ("out dstate0", g.get("dstate0"))), lens)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        if g.get(name) is None:
            g[name] = torch.empty(t.shape, dtype=t.dtype, device=dev)
        else:
            _expect("out " + name, g[name], t.dtype, t.shape, dev)
    if not want_dstate0:
        g["dstate0"] = None
    elif g.get("dstate0") is None:
        g["dstate0"] = torch.empty(shape, dtype=torch.float32, device=dev)
    if workspace is not None or need > 256:
        workspace = _workspace(workspace, need, dev)
    _streams.keep(stream, q, k, v, log_decay, state0, do, dstate, lens, workspace, *g.values())
    nat.check(_call("ssd_linattn_backward")(
        d, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(state0),
        do.data_ptr(), _ptr(dstate), _ptr(lens), g["dq"].data_ptr(), g["dk"].data_ptr(),
        g["dv"].data_ptr(), _ptr(g["dstate0"]), _ptr(workspace), _size(workspace),
        _streams.handle(stream, dev)))
    return g


def linattn_step(q, k, v, log_decay, state, *, scale=1.0, slots=None, state_out=None, out=None,
                 stream=None):
    """One token of every row: q, k [B,G,K], v [B,H,V]; log_decay [H], or
    [B,H] for decays of the token; state [rows,H,V,K] fp32.  Row b's state is
    state[slots[b]] (slots [B] int32 on the device, each row its own slot; one
    outside the state's rows marks an idle row: its o is zero and no state
    changes), or state[b] where slots is None.  The new states go to state_out
    (may be `state` itself, the default is a new tensor, or `state` itself
    with slots).  Returns (o [B,H,V], state_out).

    A step of the SSD core's recurrence is this one with v = dt x, k = B,
    q = C, log_decay = dt A, and D x added to o."""
    d = _linattn_dims(q, k, v, scale, log_decay, None, True)[0]
    dev = q.device
    _check_device(dev, stream)
    rows = state.shape[0] if state.dim() else 0
    _expect("state", state, torch.float32, (rows, d.nheads, d.dv, d.dk), dev)
    if slots is not None:
        _expect("slots", slots, torch.int32, (d.batch,), dev)
    elif rows != d.batch:
        raise ValueError(f"state: {rows} rows, expected {d.batch}")
    if state_out is None:
        state_out = torch.empty_like(state) if slots is None else state
    else:
        _expect("state_out", state_out, torch.float32, state.shape, dev)
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=dev)
    else:
        _expect("out", out, v.dtype, v.shape, dev)
    _streams.keep(stream, q, k, v, log_decay, state, slots, out, state_out)
    nat.check(_call("ssd_linattn_step")(
        d, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
        d.nheads if log_decay.dim() == 2 else 0, state.data_ptr(), state_out.data_ptr(),
        _ptr(slots), rows, out.data_ptr(), _streams.handle(stream, dev)))
    return out, state_out


# ---- norms around a block ----------------------------------------------------------

def _rows_of(name, t, shape, dtype, dev):
    """The stride of its rows: rows dense, the rows themselves evenly spaced
    (whatever the strides of extents of 1)."""
    _expect(name, t, dtype, shape, dev, False)
    width = shape[-1]
    if t.is_contiguous():
        return width
    outer = [(n, s) for n, s in zip(t.shape[:-1], t.stride()) if n > 1]
    if t.stride(-1) == 1 or width == 1:
        if not outer:
            return width
        step = outer[-1][1]
        if step >= width and all(s == n * inner for (_, s), (n, inner) in zip(outer, outer[1:])):
            return step
    raise ValueError(f"{name}: rows must be contiguous and evenly spaced")


def _block_norm_args(residual, y, z, w_post, res_scale, w_pre):
    """(rows, width, dtype codes, row strides, workspace bytes) after the checks."""
    dev = y.device
    if not y.is_cuda:
        raise ValueError("y: must be a CUDA tensor (no CPU path exists)")
    key = ["norm", y.shape, y.stride(), y.dtype]
    for t in (residual, z, w_post, res_scale, w_pre):
        if t is not None:
            if t.device != dev:
                raise ValueError(f"a tensor is on {t.device}, expected {dev}")
            key += (t.shape, t.stride(), t.dtype)
        else:
            key.append(None)
    key = tuple(key)
    got = _layouts.get(key)
    if got is not None:
        return got
    code = _io_type("y", y)
    width = y.shape[-1]
    if residual.dtype not in (y.dtype, torch.float32):
        raise TypeError(f"residual: dtype {residual.dtype}, expected {y.dtype} or torch.float32")
    _expect("residual", residual, residual.dtype, y.shape, dev)
    ys = _rows_of("y", y, y.shape, y.dtype, dev)
    zs = 0 if z is None else _rows_of("z", z, y.shape, y.dtype, dev)
    for name, w in (("w_post", w_post), ("w_pre", w_pre), ("res_scale", res_scale)):
        if w is not None:
            _expect(name, w, torch.float32, (width,), dev)
    rows = y.numel() // width if width else 0
    n = _call("ssd_block_norm_workspace_bytes")(rows, width)
    if n == 0:
        raise nat.SsdError(nat.SSD_ERR_UNSUPPORTED, nat.last_error() or "shape rejected")
    return _layouts.keep(key, (rows, width, code, _IO_TYPES[residual.dtype], ys, zs, n))


def block_norm_forward(residual, y, z, w_post, res_scale, w_pre, eps, *, want_stats=True, out=None,
                       stream=None):
    """After a block with output y: new = residual + res_scale * rmsnorm(y)
    w_post silu(z), x = rmsnorm(new) w_pre over the last dimension (up to
    8192).  z (the gate) and res_scale may be None.  y, z: fp32 or bf16, rows
    evenly spaced; residual: their type or fp32.  Weights [width] fp32.
    Returns (new residual, x, stats [..., 2] fp32 for the backward or None:
    those of y and of the residual before its rounding);
    out: dict of preallocated "residual" (may be `residual` itself), "x"."""
    rows, width, code, rcode, ys, zs, _ = _block_norm_args(residual, y, z, w_post, res_scale,
                                                           w_pre)
    dev = y.device
    _check_device(dev, stream)
    out = {} if out is None else out
    new, x = out.get("residual"), out.get("x")
    if new is None:
        new = torch.empty_like(residual)
    else:
        _expect("out residual", new, residual.dtype, y.shape, dev)
    if x is None:
        x = torch.empty(y.shape, dtype=y.dtype, device=dev)
    else:
        _expect("out x", x, y.dtype, y.shape, dev)
    stats = torch.empty(*y.shape[:-1], 2, dtype=torch.float32, device=dev) if want_stats else None
    _streams.keep(stream, residual, y, z, w_post, res_scale, w_pre, new, x, stats)
    nat.check(_call("ssd_block_norm_forward")(
        rows, width, code, rcode, residual.data_ptr(), y.data_ptr(), ys, _ptr(z), zs,
        w_post.data_ptr(), _ptr(res_scale), w_pre.data_ptr(), float(eps), new.data_ptr(),
        x.data_ptr(), _ptr(stats), _streams.handle(stream, dev)))
    return new, x, stats


def block_norm_backward(new_residual, y, z, w_post, res_scale, w_pre, eps, dx, dnew=None,
                        stats=None, *, out=None, workspace=None, stream=None):
    """Gradients of sum(dx * x) + sum(dnew * new): dict dresidual, dy, dz (None
    without z), dw_post, dres_scale, dw_pre.  new_residual is the forward's;
    stats as the forward returned them, or None (recomputed)."""
    rows, width, code, rcode, ys, zs, need = _block_norm_args(new_residual, y, z, w_post,
                                                              res_scale, w_pre)
    dev = y.device
    _check_device(dev, stream)
    _expect("dx", dx, y.dtype, y.shape, dev)
    if dnew is not None:
        _expect("dnew", dnew, new_residual.dtype, y.shape, dev)
    if stats is not None:
        _expect("stats", stats, torch.float32, (*y.shape[:-1], 2), dev)
    g = dict(out) if out is not None else {}
    for name, dt, shape in (("dresidual", new_residual.dtype, y.shape), ("dy", y.dtype, y.shape),
                            ("dz", y.dtype, y.shape), ("dw_post", torch.float32, (width,)),
                            ("dres_scale", torch.float32, (width,)),
                            ("dw_pre", torch.float32, (width,))):
        if (name == "dz" and z is None) or (name == "dres_scale" and res_scale is None):
            g[name] = None
        elif g.get(name) is None:
            g[name] = torch.empty(shape, dtype=dt, device=dev)
        else:
            _expect("out " + name, g[name], dt, shape, dev)
    workspace = _workspace(workspace, need, dev)
    _streams.keep(stream, new_residual, y, z, w_post, res_scale, w_pre, dx, dnew, stats,
                  workspace, *g.values())
    nat.check(_call("ssd_block_norm_backward")(
        rows, width, code, rcode, new_residual.data_ptr(), y.data_ptr(), ys, _ptr(z), zs,
        w_post.data_ptr(), _ptr(res_scale), w_pre.data_ptr(), float(eps), _ptr(stats),
        dx.data_ptr(), _ptr(dnew), g["dresidual"].data_ptr(), g["dy"].data_ptr(), _ptr(g["dz"]),
        g["dw_post"].data_ptr(), _ptr(g["dres_scale"]), g["dw_pre"].data_ptr(),
        workspace.data_ptr(), _size(workspace), _streams.handle(stream, dev)))
    return g


# ---- gradient clipping ---------------------------------------------------------------

_Tensor = torch.Tensor
_dtype = operator.attrgetter("dtype")

def clip_grad_norm(grads, max_norm, *, eps=1e-6, out=None, workspace=None, stream=None):
    """Scales the gradients by min(1, max_norm / (n + eps)), n the square root
    of the sum of all their squares; in place, or into the tensors of `out`
    (of the same sizes and types).  grads: contiguous CUDA tensors, fp32 and bf16
    mixed as they come, of any size; what is written must not overlap.  Returns n, a 0-d fp32 tensor on the
    device (nothing is synchronised).  A NaN in a gradient makes n and every
    gradient NaN."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    if len(outs) != n:
        raise ValueError(f"out: {len(outs)} tensors, expected {n}")
    dev = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
    # one list a property: hundreds of tensors are looked through in every call
    of = lambda f, ts: list(map(f, ts))  # noqa: E731
    dtypes = of(_dtype, grads)
    try:
        codes = [_IO_TYPES[t] for t in dtypes]
    except KeyError:
        raise TypeError("grads: fp32 and bf16 tensors only") from None
    if dev.type != "cuda" or of(_Tensor.get_device, grads) != [dev.index] * n:
        raise ValueError("grads: must be CUDA tensors on one device (no CPU path exists)")
    _check_device(dev, stream)
    if not all(map(_Tensor.is_contiguous, grads)):
        raise ValueError("grads: must be contiguous")
    sizes, at = of(_Tensor.numel, grads), of(_Tensor.data_ptr, grads)
    to = at
    if out is not None:
        if of(_dtype, outs) != dtypes:
            raise TypeError("out: another dtype than the gradient's")
        if of(_Tensor.numel, outs) != sizes or of(_Tensor.get_device, outs) != [dev.index] * n:
            raise ValueError("out: another size or device than the gradient's")
        if not all(map(_Tensor.is_contiguous, outs)):
            raise ValueError("out: must be contiguous")
        to = of(_Tensor.data_ptr, outs)
    if len(set(to)) < n:  # (tensors without elements may share an address)
        full = [p for p, size in zip(to, sizes) if size]
        if len(set(full)) < len(full):
            raise ValueError(("grads" if out is None else "out") + ": a tensor is there twice")
    flat = [0] * (4 * n)  # ssd_clip_tensor: g, out, numel, dtype (with a zero above it)
    flat[0::4], flat[1::4], flat[2::4], flat[3::4] = at, to, sizes, codes
    table = array.array("Q", flat)
    rows = table.buffer_info()[0] if n else None
    norm = torch.empty((), dtype=torch.float32, device=dev)
    need = 0
    if workspace is None:
        need = _call("ssd_clip_workspace_bytes")(rows, n)
        if need == 0:
            raise nat.SsdError(nat.SSD_ERR_INVALID_ARG, nat.last_error() or "tensors rejected")
    workspace = _workspace(workspace, need, dev)
    if stream is not None:
        _streams.keep(stream, norm, workspace, *grads, *outs)
    nat.check(_call("ssd_clip_grad_norm")(rows, n, float(max_norm), float(eps), norm.data_ptr(),
                                   workspace.data_ptr(), _size(workspace),
                                   _streams.handle(stream, dev)))
    return norm
