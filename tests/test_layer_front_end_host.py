"""The torch front ends without a GPU: which tensors a call keeps for another stream, and what every call refuses before anything is launched.
CPU tensors stand in for CUDA ones and a recorder for the library."""
import pytest
import torch

from state_space_model_analytic_gb300 import _streams, api, layer_api


class Stream:
    def __init__(self, handle, device=torch.device("cuda", 0)):
        self.cuda_stream, self.device, self.waited = handle, device, []

    def wait_stream(self, other):
        self.waited.append(other)


class Cuda:
    """What the patched torch and library saw."""

    def __init__(self):
        self.current, self.recorded, self.calls = Stream(1), [], []

    def entry(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 512
        return lambda *a: self.calls.append((name, a)) or 0

    def kept(self, t):
        return any(s.data_ptr() == t.data_ptr() for s in self.recorded)


@pytest.fixture
def cuda(monkeypatch):
    c = Cuda()
    empty = torch.empty
    dev = property(lambda t: getattr(t, "elsewhere", torch.device("cuda", 0)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.Tensor, "device", dev, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: c.recorded.append(t), raising=False)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: c.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_streams, "_raw_stream", lambda i: c.current.cuda_stream)
    monkeypatch.setattr(layer_api, "_call", c.entry)
    monkeypatch.setattr(layer_api, "_layouts", layer_api._Layouts())
    return c


def linattn(T=5):
    z = torch.zeros
    return {"q": z(2, T, 2, 16), "k": z(2, T, 2, 16), "v": z(2, T, 4, 8), "log_decay": z(4),
            "state": z(2, 4, 8, 16), "do": z(2, T, 4, 8), "dstate": z(2, 4, 8, 16),
            "lens": z(2, dtype=torch.int32)}


def norm():
    z = torch.zeros
    return {"residual": z(3, 8), "y": z(3, 8), "z": z(3, 8), "w_post": z(8), "res_scale": z(8),
            "w_pre": z(8), "dx": z(3, 8), "dnew": z(3, 8), "stats": z(3, 2)}


def calls():
    """(name, operands by name, the call on a stream)"""
    f = layer_api
    a = linattn()
    yield "forward", {n: a[n] for n in ("q", "k", "v", "log_decay", "state", "lens")}, lambda s, a=a: \
        f.linattn_forward(a["q"], a["k"], a["v"], a["log_decay"], a["state"], lens=a["lens"], stream=s)
    b = linattn()
    yield "backward", b, lambda s: f.linattn_backward(
        b["q"], b["k"], b["v"], b["log_decay"], b["state"], b["do"], b["dstate"], lens=b["lens"], stream=s)
    c = {n: t[:, 0].contiguous() if t.dim() == 4 and n in "qkv" else t for n, t in linattn().items()
         if n in ("q", "k", "v", "log_decay", "state")}
    c["slots"] = torch.zeros(2, dtype=torch.int32)
    yield "step", c, lambda s: f.linattn_step(c["q"], c["k"], c["v"], c["log_decay"], c["state"],
                                              slots=c["slots"], stream=s)
    d = norm()
    n6 = ("residual", "y", "z", "w_post", "res_scale", "w_pre")
    yield "norm_forward", {n: d[n] for n in n6}, lambda s: f.block_norm_forward(
        *(d[n] for n in n6), 1e-5, stream=s)
    e = norm()
    yield "norm_backward", e, lambda s: f.block_norm_backward(
        *(e[n] for n in n6), 1e-5, e["dx"], e["dnew"], e["stats"], stream=s)
    g = {"a": torch.zeros(3), "b": torch.zeros(4), "out a": torch.zeros(3), "out b": torch.zeros(4)}
    yield "clip", g, lambda s: f.clip_grad_norm([g["a"], g["b"]], 1.0, out=[g["out a"], g["out b"]],
                                                stream=s)


NAMES = ["forward", "backward", "step", "norm_forward", "norm_backward", "clip"]


@pytest.mark.parametrize("at", range(6), ids=NAMES)
def test_every_operand_is_kept_for_another_stream(cuda, at):
    """A temporary operand is not handed out again before the stream is done
    with it, and the call starts after the current stream's work."""
    _, operands, run = list(calls())[at]
    side = Stream(2)
    run(side)
    assert side.waited == [cuda.current] and len(cuda.calls) == 1
    assert [n for n, t in operands.items() if not cuda.kept(t)] == []


@pytest.mark.parametrize("at", range(6), ids=NAMES)
def test_nothing_is_kept_on_the_current_stream(cuda, at):
    _, _, run = list(calls())[at]
    run(None)
    run(cuda.current)
    assert not cuda.recorded and not cuda.current.waited


def core_calls():
    """(name, operands by name, the call on a stream) of the core's front end"""
    z = torch.zeros
    core = {"x": z(2, 16, 4, 16), "dt": z(2, 16, 4), "A": z(4), "B": z(2, 16, 2, 16),
            "C": z(2, 16, 2, 16), "D": z(4), "h0": z(2, 4, 16, 16)}
    raw = {"x": core["x"], "dt_raw": core["dt"], "dt_bias": z(4), "a_log": z(4),
           **{n: core[n] for n in ("B", "C", "D", "h0")}}
    more = {"dy": z(2, 16, 4, 16), "chunk_states": z(2, 1, 4, 16, 16)}
    yield "forward", core, lambda s: api.forward(*core.values(), chunk=16, stream=s)
    yield "backward", {**core, **more}, lambda s: api.backward(
        *core.values(), *more.values(), chunk=16, stream=s)
    yield "forward_raw", raw, lambda s: api.forward_raw(*raw.values(), chunk=16, stream=s)
    yield "backward_raw", {**raw, **more}, lambda s: api.backward_raw(
        *raw.values(), *more.values(), chunk=16, stream=s)
    n = {"y": z(3, 8), "z": z(3, 8), "weight": z(8), "dout": z(3, 8), "inv_rms": z(3)}
    a = [n["y"], n["z"], n["weight"], 1e-5]
    yield "rmsnorm_gated_forward", {i: n[i] for i in ("y", "z", "weight")}, lambda s: \
        api.rmsnorm_gated_forward(*a, stream=s)
    yield "rmsnorm_gated_backward", n, lambda s: api.rmsnorm_gated_backward(
        *a, n["dout"], n["inv_rms"], stream=s)
    c = {"x": z(2, 5, 8), "weight": z(8, 4), "bias": z(8), "init_state": z(2, 8, 4)}
    yield "conv1d_silu_forward", c, lambda s: api.conv1d_silu_forward(*c.values(), stream=s)
    dout = z(2, 5, 8)
    yield "conv1d_silu_backward", {**c, "dout": dout}, lambda s: api.conv1d_silu_backward(
        *c.values(), dout, stream=s)


@pytest.fixture
def core(cuda, monkeypatch):
    class Library:
        def __getattr__(self, name):
            return cuda.entry(name)
    monkeypatch.setattr(api.nat, "lib", lambda: Library())
    return cuda


EVERY = [(calls, i, n) for i, n in enumerate(NAMES)] + [(core_calls, i, n) for i, (n, _, _) in
                                                        enumerate(core_calls())]


@pytest.mark.parametrize("of,at", [e[:2] for e in EVERY], ids=[e[2] for e in EVERY])
def test_another_device_than_the_current_one_is_refused(core, monkeypatch, of, at):
    """Tensors, or a stream, of a device that the launch would not go to."""
    run = list(of())[at][-1]
    run(None)
    run(Stream(2))
    assert len(core.calls) == 2
    with pytest.raises(ValueError, match="cuda:1"):
        run(Stream(3, torch.device("cuda", 1)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for stream in (None, Stream(2)):
        with pytest.raises(ValueError, match="current device"):
            run(stream)
    assert len(core.calls) == 2


@pytest.mark.parametrize("at", range(8), ids=[n for n, _, _ in core_calls()])
def test_the_core_keeps_every_operand_too(core, at):
    _, operands, run = list(core_calls())[at]
    run(None)
    assert not core.recorded
    side = Stream(2)
    run(side)
    assert side.waited == [core.current] and len(core.calls) == 2
    assert [n for n, t in operands.items() if not core.kept(t)] == []
    # and its results: every pointer that the library was given, but the stream's
    given = {p for p in core.calls[1][1] if isinstance(p, int) and p > 1 << 20}
    assert given <= {t.data_ptr() for t in core.recorded}


@pytest.mark.parametrize("at", [0, 1, 4, 5], ids=[NAMES[i] for i in (0, 1, 4, 5)])
def test_a_workspace_that_is_not_the_device_s_is_refused(cuda, monkeypatch, at):
    """The host's memory, another device's, or memory with gaps."""
    name = ("linattn_forward", "linattn_backward", None, None, "block_norm_backward",
            "clip_grad_norm")[at]
    f = getattr(layer_api, name)
    bad = [torch.zeros(512, dtype=torch.uint8) for _ in range(2)]
    bad[0].elsewhere, bad[1].elsewhere = torch.device("cpu"), torch.device("cuda", 1)
    bad.append(torch.zeros(1024, dtype=torch.uint8)[::2])
    for w in bad:
        monkeypatch.setattr(layer_api, name, lambda *a, **k: f(*a, workspace=w, **k))
        with pytest.raises(ValueError, match="workspace"):
            list(calls())[at][-1](None)
    monkeypatch.setattr(layer_api, name, lambda *a, **k: f(*a, workspace=torch.zeros(512), **k))
    list(calls())[at][-1](None)
    assert len(cuda.calls) == 1


def test_a_scale_that_changes_in_place_is_read_in_every_call(cuda):
    """What a call keeps for the next one with the same operands' shapes goes by
    the scale's value, not by the object that holds it."""
    a, scale = linattn(), torch.tensor(0.5)
    for want in (0.5, 2.0):
        scale.fill_(want)
        layer_api.linattn_forward(a["q"], a["k"], a["v"], a["log_decay"], scale=scale)
        layer_api.linattn_backward(a["q"], a["k"], a["v"], a["log_decay"], None, a["do"], scale=scale)
        layer_api.linattn_step(*(a[n][:, 0] for n in "qkv"), a["log_decay"], a["state"], scale=scale)
        assert [c[1][0].scale for c in cuda.calls[-3:]] == [want] * 3


def test_rows_of_one_step_are_evenly_spaced(cuda):
    """The last step of every prompt: the stride of an extent of 1 is nobody's."""
    wide = torch.zeros(3, 5, 12)
    views = {"last step": (wide[:, -1:, :8], 60), "one row": (wide[1:2, 2:3, :8], 8),
             "one prompt": (wide[:1, :, :8], 12), "all": (wide[:, :, :8], 12),
             "one of each": (wide[:, None, :1, :8], 60)}
    for name, (y, stride) in views.items():
        r, w = torch.zeros(y.shape), torch.zeros(8)
        new, x, stats = layer_api.block_norm_forward(r, y, y, w, None, w, 1e-5)
        got = cuda.calls[-1][1]
        assert (got[0], got[1], got[6], got[8]) == (y.numel() // 8, 8, stride, stride), name
        layer_api.block_norm_backward(r, y, y, w, None, w, 1e-5, x, None, stats)
        got = cuda.calls[-1][1]
        assert (got[0], got[1], got[6], got[8]) == (y.numel() // 8, 8, stride, stride), name
    for y in (wide[:2, :3, :8], wide[:, :, :8].transpose(0, 1), wide[..., ::2], wide[:, :, :8][:, :1]
              .expand(3, 5, 8)):
        r, w = torch.zeros(y.shape), torch.zeros(y.shape[-1])
        with pytest.raises(ValueError, match="evenly spaced"):
            layer_api.block_norm_forward(r, y, y, w, None, w, 1e-5)


def test_a_tensor_clipped_into_twice_is_refused(cuda):
    """Two writers of one tensor race; one tensor read twice, and tensors without
    elements, do not."""
    f = layer_api.clip_grad_norm
    a, b, none = torch.ones(3), torch.ones(4), torch.ones(0)
    for kw in (dict(grads=[a, b, a]), dict(grads=[a, a], out=[b[:3], b[:3]])):
        with pytest.raises(ValueError, match="twice"):
            f(kw["grads"], 1.0, out=kw.get("out"))
    assert not cuda.calls
    f([a, none, b, none], 1.0)
    f([a, a], 1.0, out=[torch.ones(3), b[:3]])
    f([none, none], 1.0)
    assert len(cuda.calls) == 3
