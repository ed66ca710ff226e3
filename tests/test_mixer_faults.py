"""What Python callers learn of waits that ran out inside the mixer's kernels."""
import os
import sys

import pytest
import torch

from diagonal_state_space_gb300 import _native, api, init

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Lib:
    def __init__(self, code):
        self.code = code

    def s5_delta_fault(self):
        return self.code

    s5_rotary_fault = s5_delta_fault


@pytest.mark.parametrize("ask", [api.s5_delta_fault, api.s5_rotary_fault])
def test_the_flag_is_reported(monkeypatch, ask):
    for code, want in ((0, False), (1, True)):
        monkeypatch.setattr(_native, "lib", lambda: Lib(code))
        assert ask() is want
    monkeypatch.setattr(_native, "lib", lambda: Lib(-1))
    with pytest.raises(api.S5Error, match="could not be read"):
        ask()


def test_the_example_looks_at_the_flags(monkeypatch):
    import delta_mixer
    monkeypatch.setattr(_native, "lib", lambda: Lib(0))
    delta_mixer.finished()
    monkeypatch.setattr(_native, "lib", lambda: Lib(1))
    with pytest.raises(RuntimeError, match="ran out"):
        delta_mixer.finished()


@pytest.mark.gpu
def test_a_wait_that_ran_out_is_seen_from_python():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    x = torch.randn(1, 4096, 16, 128, device="cuda").bfloat16()
    pos, freq = torch.arange(4096, device="cuda")[None], torch.from_numpy(init.rotary_frequencies(128)[0]).cuda()
    lib = _native.lib()
    before = lib.s5_rotary_wait_limit(0)
    try:
        api.s5_rotary(x, pos, freq)
    finally:
        lib.s5_rotary_wait_limit(before)
    assert api.s5_rotary_fault(x.device) and not api.s5_rotary_fault() and not api.s5_delta_fault()
