"""Host check of the rotation's largest sizes."""
import ctypes

from diagonal_state_space_gb300 import _native

P = ctypes.c_void_p(1 << 20)     # aligned, never dereferenced on rejection


def test_heads_past_2_30_are_refused():
    lib = _native.lib()
    h = (1 << 30) + 2
    assert lib.s5_rotary(P, 2 * h, 0, P, P, 2, 0, 1.0, 0, 1, h, 2, P, 2 * h, None) == 2
    # refused for its address: the size itself is taken
    assert lib.s5_rotary(None, 1 << 31, 0, P, P, 2, 0, 1.0, 0, 1, 1 << 30, 2, P, 1 << 31, None) == 1
