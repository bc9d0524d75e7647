"""Host-side checks of the delta rule's and layer norm's C ABI: sizes of workspaces
and refusals, before anything touches a device."""
import ctypes

import pytest

from state_space_model_analytic_gb300 import _native as nat
from state_space_model_analytic_gb300 import build as build_lib

F = ctypes.c_void_p(1 << 20)
BAD = ctypes.c_void_p((1 << 20) + 4)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    build_lib()
    return nat.lib()


def dims(**kw):
    d = dict(batch=2, seqlen=10, nheads=4, ngroups=2, dk=16, dv=24, q_batch=320, q_step=32,
             k_batch=320, k_step=32, v_batch=960, v_step=96, dout_batch=960, dout_step=96, scale=1.0,
             dtype=nat.SSD_F32)
    d.update(kw)
    return nat.LinattnDims(**d)


def forward(L, d, q=F, la=F, be=F, s0=None, lens=None, o=F, ws=None, size=0):
    return L.ssd_delta_rule_forward(d, q, F, F, la, be, s0, lens, o, None, ws, size, None)


def backward(L, d, dout=F, la=F, be=F, dla=F, dbe=F, ws=F, size=1 << 40):
    return L.ssd_delta_rule_backward(d, F, F, F, la, be, None, dout, None, None, F, F, F, dla, dbe,
                                     None, ws, size, None)


def step(L, d, la=F, be=F, state=F, slots=None, nslots=2):
    return L.ssd_delta_rule_step(d, F, F, F, la, be, state, F, slots, nslots, F, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), nat.SSD_ERR_INVALID_ARG), (dict(seqlen=0), nat.SSD_ERR_INVALID_ARG),
    (dict(nheads=3), nat.SSD_ERR_INVALID_ARG), (dict(dtype=7), nat.SSD_ERR_INVALID_ARG),
    (dict(dk=12), nat.SSD_ERR_UNSUPPORTED), (dict(dv=136), nat.SSD_ERR_UNSUPPORTED),
    (dict(batch=70000), nat.SSD_ERR_UNSUPPORTED), (dict(seqlen=1 << 31), nat.SSD_ERR_UNSUPPORTED)])
def test_delta_dims(L, kw, code):
    d = dims(**kw)
    assert L.ssd_delta_rule_workspace_bytes(d, 0) == 0 and nat.last_error()
    assert forward(L, d) == code and nat.last_error()
    assert backward(L, d) == code and step(L, d) == code


@pytest.mark.parametrize("kw", [dict(q_step=34), dict(k_batch=2), dict(v_step=0), dict(v_batch=-960)])
def test_delta_strides(L, kw):
    assert forward(L, dims(**kw)) == nat.SSD_ERR_INVALID_ARG
    assert "strides" in nat.last_error()
    assert backward(L, dims(**kw)) == nat.SSD_ERR_INVALID_ARG


def test_delta_pointers(L):
    d = dims()
    for kw in (dict(q=None), dict(la=None), dict(be=None), dict(o=None)):
        assert forward(L, d, **kw) == nat.SSD_ERR_INVALID_ARG and "NULL" in nat.last_error()
    for kw in (dict(q=BAD), dict(s0=BAD), dict(la=ODD), dict(be=ODD), dict(lens=ODD)):
        assert forward(L, d, **kw) == nat.SSD_ERR_ALIGNMENT
    for kw in (dict(dout=None), dict(dla=None), dict(dbe=None)):
        assert backward(L, d, **kw) == nat.SSD_ERR_INVALID_ARG and "NULL" in nat.last_error()
    assert backward(L, d, dla=ODD) == nat.SSD_ERR_ALIGNMENT
    d1 = dims(seqlen=1)
    assert step(L, d) == nat.SSD_ERR_INVALID_ARG and "seqlen" in nat.last_error()
    assert step(L, d1, state=None) == nat.SSD_ERR_INVALID_ARG
    assert step(L, d1, be=None) == nat.SSD_ERR_INVALID_ARG
    assert step(L, d1, nslots=1) == nat.SSD_ERR_INVALID_ARG and "nslots" in nat.last_error()
    assert step(L, d1, slots=ODD) == nat.SSD_ERR_ALIGNMENT


def test_delta_workspace(L):
    d = dims()
    assert L.ssd_delta_rule_workspace_bytes(d, 2) == 0
    need = L.ssd_delta_rule_workspace_bytes(d, 1)
    # a state, its gradient and two rows of 24 for each of 32 steps of 8 heads, and the heads' dq, dk
    assert need >= 4 * 8 * (2 * 24 * 16 + 2 * 32 * 24) + 4 * 2 * 2 * 10 * 4 * 16
    assert backward(L, d, ws=None) == nat.SSD_ERR_INVALID_ARG
    assert backward(L, d, size=need - 1) == nat.SSD_ERR_INVALID_ARG and "workspace" in nat.last_error()
    assert backward(L, d, ws=BAD, size=need) == nat.SSD_ERR_ALIGNMENT
    # sizes pass 32 bits
    big = dims(batch=16, seqlen=1 << 20, nheads=64, ngroups=64, dk=128, dv=128, dtype=nat.SSD_BF16)
    assert L.ssd_delta_rule_workspace_bytes(big, 1) > 1 << 41


def ln_forward(L, rows=4, width=64, dtype=nat.SSD_F32, x=F, stride=64, w=F, eps=1e-5, y=F, stats=None):
    return L.ssd_layer_norm_forward(rows, width, dtype, x, stride, w, None, eps, y, stats, None)


def ln_backward(L, rows=4, width=64, dtype=nat.SSD_F32, x=F, stride=64, eps=1e-5, dy=F, dx=F, dw=F,
                ws=F, size=1 << 30):
    return L.ssd_layer_norm_backward(rows, width, dtype, x, stride, None, eps, None, dy, dx, dw, None,
                                     ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), nat.SSD_ERR_INVALID_ARG), (dict(dtype=5), nat.SSD_ERR_INVALID_ARG),
    (dict(width=8193, stride=8193), nat.SSD_ERR_UNSUPPORTED), (dict(stride=63), nat.SSD_ERR_INVALID_ARG),
    (dict(eps=-1.0), nat.SSD_ERR_INVALID_ARG), (dict(eps=float("nan")), nat.SSD_ERR_INVALID_ARG),
    (dict(x=None), nat.SSD_ERR_INVALID_ARG), (dict(x=ODD), nat.SSD_ERR_ALIGNMENT)])
def test_layer_norm(L, kw, code):
    assert ln_forward(L, **kw) == code and nat.last_error()
    assert ln_backward(L, **kw) == code


def test_layer_norm_pointers_and_workspace(L):
    assert ln_forward(L, y=None) == nat.SSD_ERR_INVALID_ARG
    assert ln_forward(L, w=ODD) == nat.SSD_ERR_ALIGNMENT
    assert ln_forward(L, stats=BAD) == nat.SSD_ERR_ALIGNMENT
    assert ln_backward(L, dy=None) == nat.SSD_ERR_INVALID_ARG
    assert ln_backward(L, dx=None) == nat.SSD_ERR_INVALID_ARG
    assert ln_backward(L, dw=ODD) == nat.SSD_ERR_ALIGNMENT
    need = L.ssd_layer_norm_workspace_bytes(4, 64)
    assert ln_backward(L, size=need - 1) == nat.SSD_ERR_INVALID_ARG
    assert ln_backward(L, ws=BAD) == nat.SSD_ERR_ALIGNMENT
    assert L.ssd_layer_norm_workspace_bytes(0, 64) == 0 and L.ssd_layer_norm_workspace_bytes(4, 8193) == 0
