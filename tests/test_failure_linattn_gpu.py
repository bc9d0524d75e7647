"""Failure detection of the linear-attention kernels on the GPU without a fault:
their bounded wait runs out on a barrier that nothing completes, a second warp
follows it, and the host reads which wait it was."""
import re

import pytest

pytestmark = pytest.mark.gpu


def test_the_walk_s_wait_runs_out_and_is_reported():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import state_space_model_analytic_gb300 as ssd
    from state_space_model_analytic_gb300 import _native as nat
    ssd.build()
    L = nat.lib()
    nat.check(L.ssd_device_status())  # clear anything left over
    nat.check(L.ssd_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream or None))
    torch.cuda.synchronize()
    assert L.ssd_device_status() == nat.SSD_ERR_DEVICE_TIMEOUT
    flag = int(re.search(r"flag 0x([0-9a-f]+)", nat.last_error()).group(1), 16)
    assert flag & 0xff and flag >> 24 == 1
    assert L.ssd_device_status() == nat.SSD_OK
    # the walks run as before
    q = torch.randn(1, 300, 2, 64, device="cuda").bfloat16()
    la = torch.full((2,), -0.1, device="cuda")
    a, b = ssd.linattn_forward(q, q, q, la), ssd.linattn_forward(q, q, q, la)
    assert torch.isfinite(a[0]).all() and all(torch.equal(x, y) for x, y in zip(a, b))
    assert L.ssd_device_status() == nat.SSD_OK
