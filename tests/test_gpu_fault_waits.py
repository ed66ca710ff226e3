"""GPU test that the questions whether a wait ran out wait for the device, streams that do not block the default one among
them: an answer before the kernels end would call results valid that are not."""
import pytest
import torch

from diagonal_state_space_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ask", [api.s5_gated_scan_fault, api.s5_rotary_fault, api.s5_delta_fault], ids=lambda f: f.__name__)
def test_the_answer_waits_for_other_streams(ask):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    assert not ask()                     # loaded, and nothing is left over
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)   # clocks: about 0.2 s
    assert not side.query()
    assert not ask()
    assert side.query()
