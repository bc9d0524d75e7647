"""GPU parity of gradient clipping against the float64 reference.

Tolerances: a thread adds at most a few hundred squares in fp32 and the rest
in fp64, so n is within 2^-15 relative (256 roundings of 2^-24, halved by the
root, and its own); out = c g adds two roundings in fp32, one of at most 2^-8 in
bf16."""
import numpy as np
import pytest

from oracle import layer
from state_space_model_analytic_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from state_space_model_analytic_gb300 import build
    build()


def make(sizes, kinds, std=1.0, seed=0, pad=0):
    """Host values and device tensors: views of one buffer a type, `pad`
    elements apart (odd offsets)."""
    import torch
    rng = np.random.default_rng(seed)
    vals = [synth.round_to(std * rng.standard_normal(n), k) for n, k in zip(sizes, kinds)]
    ts = []
    for v, k in zip(vals, kinds):
        flat = torch.zeros(v.size + pad + 8, dtype=torch.bfloat16 if k == "bf16" else torch.float32,
                           device="cuda")
        t = flat[pad:pad + v.size]
        t.copy_(torch.from_numpy(v.astype(np.float32)))
        ts.append(t)
    return vals, ts


def close(t, ref, kind):
    got = t.double().cpu().numpy().reshape(-1)
    bound = (2.0 ** -8 if kind == "bf16" else 0) * np.abs(ref) * 1.01 + 2.0 ** -14 * np.abs(ref) + 1e-38
    if kind == "bf16":
        bound = bound + 1e-38
    assert (np.abs(got - ref) <= bound).all(), float(np.abs(got - ref).max())


SIZES = [[1], [5, 1, 9], [4096, 4097, 3], [100000, 7, 0, 65536, 33], [2000001]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_out_of_place_and_in_place(sizes, kind, pad):
    import torch
    import state_space_model_analytic_gb300 as ssd
    kinds = [("bf16", "f32")[i % 2] if kind == "mixed" else kind for i in range(len(sizes))]
    vals, ts = make(sizes, kinds, seed=len(sizes), pad=pad)
    n_ref, out_ref = layer.clip(vals, 0.75, 1e-6)
    outs = [torch.full_like(t, 7.0) for t in ts]  # aligned differently from t
    keep = [t.clone() for t in ts]
    n = ssd.clip_grad_norm(ts, 0.75, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    assert abs(float(n) - n_ref) <= 2.0 ** -15 * n_ref
    for t, r, k in zip(outs, out_ref, kinds):
        close(t, r, k)
    n2 = ssd.clip_grad_norm(ts, 0.75)
    assert torch.equal(n, n2)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_below_the_limit_nothing_changes():
    import torch
    import state_space_model_analytic_gb300 as ssd
    vals, ts = make([1000, 17], ["f32", "bf16"], 0.01)
    keep = [t.clone() for t in ts]
    outs = [torch.zeros_like(t) for t in ts]
    for limit in (1e3, float("inf")):
        ssd.clip_grad_norm(ts, limit, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(ts, outs))
        ssd.clip_grad_norm(ts, limit)
        assert all(torch.equal(a, b) for a, b in zip(ts, keep))


def test_many_tensors_and_slices_of_memory():
    """More tensors than one launch's table holds; the memory between them is
    not touched."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    flat = torch.randn(2500 * 40, device="cuda")
    views = [flat[i * 40 + 3:i * 40 + 3 + i % 30] for i in range(2500)]
    mask = torch.zeros_like(flat, dtype=torch.bool)
    for i in range(2500):
        mask[i * 40 + 3:i * 40 + 3 + i % 30] = True
    was = flat.clone()
    n_ref = float(was[mask].double().norm())
    n = ssd.clip_grad_norm(views, 1.0)
    assert abs(float(n) - n_ref) <= 2.0 ** -15 * n_ref
    assert torch.equal(flat[~mask], was[~mask])
    err = (flat[mask].double() - was[mask].double() / (n_ref + 1e-6)).abs()
    assert bool((err <= 2.0 ** -14 * was[mask].double().abs() / n_ref).all())


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e15, 1e30])
def test_magnitudes_whose_squares_leave_fp32(std):
    import state_space_model_analytic_gb300 as ssd
    for kind in ("f32", "bf16"):
        vals, ts = make([5000, 3], [kind, kind], std)
        n_ref, out_ref = layer.clip(vals, std, 0.0)
        n = ssd.clip_grad_norm(ts, std, eps=0.0)
        assert abs(float(n) - n_ref) <= 2.0 ** -15 * n_ref
        for t, r in zip(ts, out_ref):
            close(t, r, kind)


def test_zeros_nan_inf_and_no_tensors():
    import torch
    import state_space_model_analytic_gb300 as ssd
    z = torch.zeros(100, device="cuda")
    for eps in (0.0, 1e-6):
        assert float(ssd.clip_grad_norm([z], 1.0, eps=eps)) == 0.0 and not z.any()
    a, b = torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)
    a[3] = float("inf")
    n = ssd.clip_grad_norm([a, b], 1.0)
    assert torch.isinf(n) and torch.isnan(a[3]) and not b.any() and not a[:3].any()
    a, b = torch.ones(100, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)
    a[3] = float("nan")
    n = ssd.clip_grad_norm([a, b], 1.0)
    assert torch.isnan(n) and torch.isnan(a).all() and torch.isnan(b).all()
    assert float(ssd.clip_grad_norm([], 1.0)) == 0.0
    assert float(ssd.clip_grad_norm([z[:0]], 1.0)) == 0.0
    a = torch.ones(4, device="cuda")
    ssd.clip_grad_norm([a], 0.0)
    assert not a.any()


def test_equal_runs_on_another_stream():
    import torch
    import state_space_model_analytic_gb300 as ssd
    _, ts = make([3000000, 4095, 1000001], ["bf16", "f32", "f32"])
    o1, o2 = [torch.empty_like(t) for t in ts], [torch.empty_like(t) for t in ts]
    n1 = ssd.clip_grad_norm(ts, 1.0, out=o1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n2 = ssd.clip_grad_norm(ts, 1.0, out=o2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n1, n2) and all(torch.equal(a, b) for a, b in zip(o1, o2))


def test_another_stream_starts_after_the_current_one():
    """The call's memory comes from the current stream's allocator, whose earlier
    work may still use it: here that work also writes the gradients."""
    import torch
    import state_space_model_analytic_gb300 as ssd
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    ts = [torch.zeros(1000, device="cuda") for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        big.fill_(i)
    for t in ts:
        t.fill_(2.0)
    n = ssd.clip_grad_norm(ts, 1e9, stream=side)
    torch.cuda.synchronize()
    assert abs(float(n) - 2 * 3000 ** 0.5) < 1e-4


def test_refusals():
    import torch
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    g = torch.ones(10, device="cuda")
    with pytest.raises(nat.SsdError):
        ssd.clip_grad_norm([g], -1.0)
    with pytest.raises(nat.SsdError):
        ssd.clip_grad_norm([g], float("nan"))
    with pytest.raises(nat.SsdError):
        ssd.clip_grad_norm([g], 1.0, eps=-1.0)
    with pytest.raises(TypeError):
        ssd.clip_grad_norm([g.half()], 1.0)
    with pytest.raises(ValueError):
        ssd.clip_grad_norm([g.cpu()], 1.0)
    with pytest.raises(ValueError):
        ssd.clip_grad_norm([torch.ones(4, 4, device="cuda").t()], 1.0)
    with pytest.raises(ValueError):
        ssd.clip_grad_norm([g], 1.0, out=[g[:5]])
    with pytest.raises(TypeError):
        ssd.clip_grad_norm([g], 1.0, out=[g.bfloat16()])
    with pytest.raises(ValueError):
        ssd.clip_grad_norm([g, g], 1.0, out=[g])
    with pytest.raises(nat.SsdError):
        ssd.clip_grad_norm([g], 1.0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
