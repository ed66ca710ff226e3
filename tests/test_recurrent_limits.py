"""Host checks of the largest sizes of the gated recurrence and the short convolution: channel counts whose blocks would end
past a 32-bit integer are refused, and what is said of buffers at the largest that are not."""
import ctypes

import pytest

from diagonal_state_space_gb300 import _native, build

UNSUP, MOST, FIRST = 2, 2 ** 31 - 256, 2 ** 31 - 255
P, Q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)   # aligned, never dereferenced on rejection


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.lib()


@pytest.mark.parametrize("C", [FIRST, 2 ** 31 - 64, 2 ** 31 - 8, 2 ** 31 - 1])
def test_channels_past_the_largest_are_refused(lib, C):
    assert lib.s5_gated_scan_saved_size(1, 1, C) == 0 and lib.s5_gated_scan_workspace_size(1, 1, C) == 0
    assert lib.s5_short_conv_workspace_size(C, 4) == 0
    assert lib.s5_gated_scan_forward(P, C, P, C, P, C, 0, P, None, None, None, 1, 1, 1, C, Q, C, None, None, 0, None) == UNSUP
    big = 1 << 62
    assert lib.s5_gated_scan_backward(P, C, P, C, P, C, 0, P, None, None, 1, 1, 1, C, P, C, None, P, big, Q, C, Q, C, Q, C, Q, None, P, big,
                                      None) == UNSUP
    assert lib.s5_short_conv_forward(P, C, 0, P, None, 0, None, None, None, 1, 1, C, 4, Q, C, None, None) == UNSUP
    assert lib.s5_short_conv_backward(P, C, 0, P, None, 0, None, None, None, 1, 1, C, 4, P, C, None, Q, C, Q, None, None, P, big, None) == UNSUP
    assert lib.s5_short_conv_step(P, 0, P, None, 0, 1, C, 4, Q, Q, None) == UNSUP


def test_buffers_of_the_largest(lib):
    assert lib.s5_gated_scan_saved_size(1, 33, MOST) == 256 + 4 * 2 * MOST
    assert lib.s5_gated_scan_workspace_size(1, 1, MOST) >= 4 * MOST
    assert lib.s5_short_conv_workspace_size(MOST, 2) >= 4 * 3 * MOST
