"""The torch front end of the delta rule and layer norm without a GPU: which tensors a
call keeps for another stream, and what is refused before anything is launched (as
test_layer_front_end_host.py does for the other layer operators)."""
import pytest
import torch

from state_space_model_analytic_gb300 import layer_api
from test_layer_front_end_host import Stream, cuda  # noqa: F401


def delta(T=5):
    z = torch.zeros
    return {"q": z(2, T, 2, 16), "k": z(2, T, 2, 16), "v": z(2, T, 4, 8), "log_decay": z(2, T, 4),
            "beta": z(2, T, 4), "state": z(2, 4, 8, 16), "do": z(2, T, 4, 8), "dstate": z(2, 4, 8, 16),
            "lens": z(2, dtype=torch.int32)}


def token():
    a = delta()
    c = {n: a[n][:, 0].contiguous() for n in ("q", "k", "v", "log_decay", "beta")}
    return {**c, "state": a["state"], "slots": torch.zeros(2, dtype=torch.int32)}


def calls():
    """(name, operands by name, the call on a stream)"""
    f = layer_api
    a, b, c = delta(), delta(), token()
    five = ("q", "k", "v", "log_decay", "beta")
    yield "forward", {n: a[n] for n in five + ("state", "lens")}, lambda s, **k: f.delta_rule_forward(
        *(a[n] for n in five), a["state"], lens=a["lens"], stream=s, **k)
    yield "backward", b, lambda s, **k: f.delta_rule_backward(
        *(b[n] for n in five), b["state"], b["do"], b["dstate"], lens=b["lens"], stream=s, **k)
    yield "step", c, lambda s, **k: f.delta_rule_step(*(c[n] for n in five), c["state"], slots=c["slots"],
                                                      stream=s, **k)
    x = {"x": torch.zeros(3, 8), "weight": torch.zeros(8), "bias": torch.zeros(8)}
    yield "norm_forward", x, lambda s, **k: f.layer_norm_forward(*x.values(), 1e-5, stream=s, **k)
    y = {"x": torch.zeros(3, 8), "weight": torch.zeros(8), "dy": torch.zeros(3, 8), "stats": torch.zeros(3, 2)}
    yield "norm_backward", y, lambda s, **k: f.layer_norm_backward(
        y["x"], y["weight"], y["dy"], 1e-5, y["stats"], stream=s, **k)


NAMES = ["forward", "backward", "step", "norm_forward", "norm_backward"]


@pytest.mark.parametrize("at", range(5), ids=NAMES)
def test_operands_and_results_are_kept_for_another_stream_alone(cuda, at):  # noqa: F811
    _, operands, run = list(calls())[at]
    run(None)
    run(cuda.current)
    assert not cuda.recorded and not cuda.current.waited
    side = Stream(2)
    run(side)
    assert side.waited == [cuda.current] and len(cuda.calls) == 3
    assert [n for n, t in operands.items() if not cuda.kept(t)] == []
    given = {p for p in cuda.calls[2][1] if isinstance(p, int) and p > 1 << 20}
    assert given <= {t.data_ptr() for t in cuda.recorded}


@pytest.mark.parametrize("at", range(5), ids=NAMES)
def test_another_device_is_refused(cuda, monkeypatch, at):  # noqa: F811
    _, operands, run = list(calls())[at]
    run(None)
    with pytest.raises(ValueError, match="cuda:1"):
        run(Stream(3, torch.device("cuda", 1)))
    for n, t in operands.items():  # one tensor elsewhere, also after a call with the same shapes
        t.elsewhere = torch.device("cuda", 1)
        with pytest.raises(ValueError):
            run(None)
        del t.elsewhere
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        run(None)
    assert len(cuda.calls) == 1


@pytest.mark.parametrize("at", [0, 1, 4], ids=[NAMES[i] for i in (0, 1, 4)])
def test_a_workspace_that_is_not_the_device_s_is_refused(cuda, at):  # noqa: F811
    run = list(calls())[at][-1]
    bad = [torch.zeros(512, dtype=torch.uint8) for _ in range(2)]
    bad[0].elsewhere, bad[1].elsewhere = torch.device("cpu"), torch.device("cuda", 1)
    for w in bad + [torch.zeros(1024, dtype=torch.uint8)[::2]]:
        with pytest.raises(ValueError, match="workspace"):
            run(None, workspace=w)
    run(None, workspace=torch.zeros(512))
    assert len(cuda.calls) == 1


def test_a_scale_that_changes_in_place_is_read_in_every_call(cuda):  # noqa: F811
    a, t, scale = delta(), token(), torch.tensor(0.5)
    five = ("q", "k", "v", "log_decay", "beta")
    for want in (0.5, 2.0):
        scale.fill_(want)
        layer_api.delta_rule_forward(*(a[n] for n in five), scale=scale)
        layer_api.delta_rule_backward(*(a[n] for n in five), None, a["do"], scale=scale)
        layer_api.delta_rule_step(*(t[n] for n in five), t["state"], scale=scale)
        assert [c[1][0].scale for c in cuda.calls[-3:]] == [want] * 3


def test_a_step_s_checks_do_not_go_by_an_earlier_call(cuda):  # noqa: F811
    """Every property that is checked is looked at again."""
    t = token()
    five = [t[n] for n in ("q", "k", "v", "log_decay", "beta")]
    run = layer_api.delta_rule_step
    run(*five, t["state"])
    z = torch.zeros
    for kw in (dict(state=z(3, 4, 8, 16)), dict(state=z(2, 4, 16, 8)), dict(state=z(2, 4, 16, 8).mT),
               dict(state=t["state"].double()), dict(state_out=z(2, 4, 8, 8)), dict(out=z(2, 4, 16)),
               dict(slots=z(3, dtype=torch.int32)), dict(slots=z(2)), dict(beta=z(2, 4).double()),
               dict(beta=z(4)), dict(log_decay=z(4, 2).t()), dict(k=z(2, 2, 8))):
        a = dict(zip(("q", "k", "v", "log_decay", "beta"), five), state=t["state"], **{})
        a.update(kw)
        for _ in range(2):
            with pytest.raises((ValueError, TypeError)):
                run(**a)
    run(*five, t["state"])
    assert len(cuda.calls) == 2


def test_rows_of_a_norm_are_evenly_spaced(cuda):  # noqa: F811
    wide = torch.zeros(3, 5, 12)
    views = {"last step": (wide[:, -1:, :8], 60), "one row": (wide[1:2, 2:3, :8], 8),
             "one prompt": (wide[:1, :, :8], 12), "all": (wide[:, :, :8], 12)}
    for name, (x, stride) in views.items():
        y, stats = layer_api.layer_norm_forward(x, None, None, 1e-5)
        got = cuda.calls[-1][1]
        assert (got[0], got[1], got[4]) == (x.numel() // 8, 8, stride), name
        layer_api.layer_norm_backward(x, None, y, 1e-5, stats)
        got = cuda.calls[-1][1]
        assert (got[0], got[1], got[4]) == (x.numel() // 8, 8, stride), name
    for x in (wide[:2, :3, :8], wide[:, :, :8].transpose(0, 1), wide[..., ::2]):
        with pytest.raises(ValueError, match="evenly spaced"):
            layer_api.layer_norm_forward(x, None, None, 1e-5)


def test_wanted_gradients_alone(cuda):  # noqa: F811
    x = torch.zeros(3, 8)
    g = layer_api.layer_norm_backward(x, None, x, 1e-5, want_dweight=False, want_dbias=False)
    assert g["dweight"] is None and g["dbias"] is None and cuda.calls[-1][1][10:12] == (None, None)
    a = delta()
    g = layer_api.delta_rule_backward(*(a[n] for n in ("q", "k", "v", "log_decay", "beta")), None, a["do"],
                                      want_dstate0=False)
    assert g["dstate0"] is None
