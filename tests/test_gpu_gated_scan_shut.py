"""GPU tests of the gated recurrence with gates nearly shut: 1 - a^2 at the end of 32 bits, value by value, and where it has
left them the same in both directions."""
import pytest
import torch

from _recurrent_gpu import TYPES
from test_gpu_gated_scan import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


# sigmoid(-86.5) is 2.7e-38, and 1 - a^2 twice that times the rate: the smallest normal value is 1.2e-38
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("C", [40, 41])
@pytest.mark.parametrize("gate,rate", [(-86.5, 1.0), (-86.5, 0.25), (-85.0, 1.0), (-80.0, 0.001), (-86.5, 8.0)])
def test_the_root_is_the_same_in_both_directions(gate, rate, C, gated, kind):
    t = make(2, 70, C, kind, gated=gated, h0=True, seed=C)
    t["ga"].fill_(gate)
    t["rate"].fill_(rate)
    check(t)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", [40, 41])
def test_a_root_that_vanishes_has_no_slope(C, kind):
    """1 - a^2 of 1.8e-39: the state is held, and what was not added has no gradient."""
    t = make(2, 70, C, kind, h0=True, seed=C)
    t["ga"].fill_(-83.0)
    t["rate"].fill_(1e-3)
    got = run(t)
    assert torch.equal(got["h_last"], t["h0"])
    for n in ("dx", "dgate_x"):
        assert torch.count_nonzero(got[n]) == 0, n
    assert got["dgate_a"].abs().max() < 1e-36
