"""Further host-side checks of the layer operators' C ABI, before anything
touches a device."""
import ctypes

from state_space_model_analytic_gb300 import _native as nat
from test_abi_layer_host import F, L, dims  # noqa: F401


def test_linattn_small_pointers_are_aligned_to_their_elements(L):
    """log_decay, lens and slots: slices of an array are taken, other addresses
    are refused before a launch."""
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731
    fd, sd = dims(), dims(seqlen=1)
    fwd = lambda la, lens: L.ssd_linattn_forward(  # noqa: E731
        fd, F, F, F, la, None, lens, F, None, F, 1 << 30, None)
    bwd = lambda la, lens: L.ssd_linattn_backward(  # noqa: E731
        fd, F, F, F, la, None, F, None, lens, F, F, F, None, F, 1 << 30, None)
    one = lambda la, slots: L.ssd_linattn_step(  # noqa: E731
        sd, F, F, F, la, 0, F, F, slots, 2, F, None)
    for call, name in ((fwd, "lens"), (bwd, "lens"), (one, "slots")):
        for n in (1, 2, 3, 6):
            assert call(at(n), None) == nat.SSD_ERR_ALIGNMENT and "log_decay" in nat.last_error()
            assert call(F, at(n)) == nat.SSD_ERR_ALIGNMENT and name in nat.last_error()
