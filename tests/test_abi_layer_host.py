"""Host-side checks of the layer operators' C ABI: sizes of workspaces and
refusals, before anything touches a device."""
import array
import ctypes

import pytest

from state_space_model_analytic_gb300 import _native as nat
from state_space_model_analytic_gb300 import build as build_lib

F = ctypes.c_void_p(1 << 20)
BAD = ctypes.c_void_p((1 << 20) + 4)


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


def forward(L, d, q=F, ws=1 << 30):
    return L.ssd_linattn_forward(d, q, F, F, F, None, None, F, None, F, ws, None)


def backward(L, d, dout=F, ws=1 << 30):
    return L.ssd_linattn_backward(d, F, F, F, F, None, dout, None, None, F, F, F, None, F, ws, None)


def step(L, d, state=F, slots=None, nslots=2, decay_batch=0):
    return L.ssd_linattn_step(d, F, F, F, F, decay_batch, state, F, slots, nslots, F, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), nat.SSD_ERR_INVALID_ARG), (dict(seqlen=0), nat.SSD_ERR_INVALID_ARG),
    (dict(nheads=3), nat.SSD_ERR_INVALID_ARG), (dict(dtype=7), nat.SSD_ERR_INVALID_ARG),
    (dict(dk=12), nat.SSD_ERR_UNSUPPORTED), (dict(dv=136), nat.SSD_ERR_UNSUPPORTED),
    (dict(batch=70000), nat.SSD_ERR_UNSUPPORTED), (dict(seqlen=1 << 31), nat.SSD_ERR_UNSUPPORTED)])
def test_linattn_dims(L, kw, code):
    d = dims(**kw)
    assert L.ssd_linattn_workspace_bytes(d, 0) == 0 and nat.last_error()
    assert forward(L, d) == code and nat.last_error()
    assert backward(L, d) == code


@pytest.mark.parametrize("kw", [dict(q_step=34), dict(k_batch=2), dict(v_step=0), dict(v_batch=-960)])
def test_linattn_strides(L, kw):
    assert forward(L, dims(**kw)) == nat.SSD_ERR_INVALID_ARG
    assert "strides" in nat.last_error()


def test_linattn_pointers_and_workspace(L):
    d = dims()
    assert forward(L, d, q=None) == nat.SSD_ERR_INVALID_ARG
    assert forward(L, d, q=BAD) == nat.SSD_ERR_ALIGNMENT
    assert backward(L, d, dout=None) == nat.SSD_ERR_INVALID_ARG
    need = L.ssd_linattn_workspace_bytes(d, 1)
    # the heads of a group are summed from fp32 parts in the workspace
    assert need >= 2 * 10 * 4 * 16 * 4 and L.ssd_linattn_workspace_bytes(d, 0) < need
    assert backward(L, d, ws=need - 1) == nat.SSD_ERR_INVALID_ARG
    assert L.ssd_linattn_workspace_bytes(d, 2) == 0
    assert L.ssd_linattn_workspace_bytes(dims(batch=64, v_batch=960), 0) == 256  # none is used
    assert L.ssd_linattn_forward(None, F, F, F, F, None, None, F, None, F, 1 << 30, None) == \
        nat.SSD_ERR_INVALID_ARG


def test_linattn_step(L):
    d = dims(seqlen=1)
    assert step(L, dims()) == nat.SSD_ERR_INVALID_ARG        # more than one step
    assert step(L, d, state=None) == nat.SSD_ERR_INVALID_ARG
    assert step(L, d, state=BAD) == nat.SSD_ERR_ALIGNMENT
    assert step(L, d, nslots=1) == nat.SSD_ERR_INVALID_ARG   # fewer states than rows
    assert step(L, d, slots=F, nslots=0) == nat.SSD_ERR_INVALID_ARG
    assert step(L, d, decay_batch=3) == nat.SSD_ERR_INVALID_ARG


def norm_forward(L, rows=4, width=64, dtype=0, res=0, y=F, ys=64, eps=1e-5):
    return L.ssd_block_norm_forward(rows, width, dtype, res, F, y, ys, None, 0, F, None, F, eps, F,
                                    F, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), nat.SSD_ERR_INVALID_ARG), (dict(width=0), nat.SSD_ERR_UNSUPPORTED),
    (dict(width=8193, ys=8193), nat.SSD_ERR_UNSUPPORTED), (dict(dtype=2), nat.SSD_ERR_INVALID_ARG),
    (dict(dtype=0, res=1), nat.SSD_ERR_INVALID_ARG), (dict(ys=63), nat.SSD_ERR_INVALID_ARG),
    (dict(eps=-1.0), nat.SSD_ERR_INVALID_ARG), (dict(eps=float("nan")), nat.SSD_ERR_INVALID_ARG),
    (dict(y=None), nat.SSD_ERR_INVALID_ARG),
    (dict(y=ctypes.c_void_p((1 << 20) + 2)), nat.SSD_ERR_ALIGNMENT)])
def test_block_norm(L, kw, code):
    assert norm_forward(L, **kw) == code and nat.last_error()


def test_block_norm_workspace(L):
    assert L.ssd_block_norm_workspace_bytes(0, 64) == 0
    assert L.ssd_block_norm_workspace_bytes(4, 8193) == 0
    need = L.ssd_block_norm_workspace_bytes(4, 64)
    assert need > 0
    args = [4, 64, 0, 0, F, F, 64, None, 0, F, None, F, 1e-5, None, F, None, F, F, None, F, None, F]
    call = L.ssd_block_norm_backward
    assert call(*args, F, need - 1, None) == nat.SSD_ERR_INVALID_ARG
    assert call(*args, None, need, None) == nat.SSD_ERR_INVALID_ARG
    assert call(*args, ctypes.c_void_p((1 << 20) + 16), need, None) == nat.SSD_ERR_ALIGNMENT


def clip(L, rows, max_norm=1.0, eps=0.0, norm=F, ws=F, bytes_=1 << 20):
    t = array.array("q", [x for r in rows for x in r])
    at = t.buffer_info()[0] if rows else None
    return (L.ssd_clip_grad_norm(at, len(rows), max_norm, eps, norm, ws, bytes_, None),
            L.ssd_clip_workspace_bytes(at, len(rows)))


@pytest.mark.parametrize("row,code", [
    ((1 << 20, 1 << 20, -1, 0), nat.SSD_ERR_INVALID_ARG), ((1 << 20, 1 << 20, 4, 2), nat.SSD_ERR_INVALID_ARG),
    ((1 << 20, 1 << 20, 4, 1 << 32), nat.SSD_ERR_INVALID_ARG),  # the reserved half
    ((0, 1 << 20, 4, 0), nat.SSD_ERR_INVALID_ARG), ((1 << 20, 0, 4, 0), nat.SSD_ERR_INVALID_ARG),
    (((1 << 20) + 2, 1 << 20, 4, 0), nat.SSD_ERR_ALIGNMENT),
    (((1 << 20) + 1, 1 << 20, 4, 1), nat.SSD_ERR_ALIGNMENT)])
def test_clip_rejects_tensors(L, row, code):
    rc, need = clip(L, [row])
    assert rc == code and need == 0 and "tensor 0" in nat.last_error()


def test_clip_arguments(L):
    good = [(1 << 20, 1 << 20, 4, 1)]
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(norm=None),
               dict(ws=None), dict(bytes_=8)):
        assert clip(L, good, **kw)[0] == nat.SSD_ERR_INVALID_ARG, kw
    assert clip(L, good, ws=ctypes.c_void_p((1 << 20) + 16))[0] == nat.SSD_ERR_ALIGNMENT
    assert L.ssd_clip_workspace_bytes(None, -1) == 0 and L.ssd_clip_workspace_bytes(None, 0) > 0
