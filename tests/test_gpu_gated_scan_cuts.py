"""GPU tests of where the gated recurrence cuts: at resets, and nowhere else.  A decay that vanishes in 32 bits is a number:
what is not finite stays so behind it until a reset, whether resets are given or not and wherever tiles begin."""
import pytest
import torch

from _recurrent_gpu import TYPES, same
from test_gpu_gated_scan import make, run

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
WIDTHS = [40, 42, 41]


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def strong(L, C, kind, rate, seed=1):
    """Decays that a few tokens multiply to less than a 32-bit value holds (rate 30), or a single one (rate 1e3)."""
    t = make(2, L, C, kind, h0=True, seed=seed)
    t["rate"].fill_(rate)
    t["ga"].fill_(2.0)
    return t


def alike(a, b):
    return all(torch.equal(a[n].nan_to_num(0.5), b[n].nan_to_num(0.5)) and torch.equal(a[n].isnan(), b[n].isnan()) for n in a)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("rate", [30.0, 1e3])
@pytest.mark.parametrize("what", [NAN, INF])
def test_resets_elsewhere_change_nothing(what, rate, C, kind):
    t = strong(700, C, kind, rate)
    t["x"][0, 37], t["dh"][1, 411] = what, what
    without = run(t)
    t["reset"] = torch.zeros(2, 700, dtype=torch.bool, device="cuda")
    assert alike(run(t), without)
    t["reset"][1, 699] = True          # the other row's end: a tile with a reset
    got = run(t)
    assert torch.equal(got["h"][0].isnan(), without["h"][0].isnan()) and torch.equal(got["h_last"][0].isnan(), without["h_last"][0].isnan())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("rate", [30.0, 1e3])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("what", [NAN, INF])
def test_what_is_not_finite_stays_until_a_reset(what, resets, rate, C, kind):
    """In the row and its last tile, which ends inside the row or is cut by its length, in the state and in the gradients."""
    t = strong(300, C, kind, rate)
    t["lengths"] = torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    t["x"][:, 37] = what
    if resets:
        t["reset"] = torch.zeros(2, 300, dtype=torch.bool, device="cuda")
        t["reset"][:, 220] = True
    got = run(t)
    end = 220 if resets else 290
    assert torch.isfinite(got["h"][:, :37]).all() and not torch.isfinite(got["h"][:, 37:end]).any()
    if resets:
        assert torch.isfinite(got["h"][:, 220:]).all() and torch.isfinite(got["h_last"]).all()
    else:
        assert not torch.isfinite(got["h_last"]).any()
    t = strong(300, C, kind, rate)
    t["lengths"] = torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    if resets:
        t["reset"] = torch.zeros(2, 300, dtype=torch.bool, device="cuda")
        t["reset"][:, 100] = True
    t["dh"][:, 250] = what
    got = run(t)
    first = 100 if resets else 0
    assert torch.isfinite(got["dx"][:, 251:]).all() and not torch.isfinite(got["dx"][:, first:251]).any()
    if resets:
        assert torch.isfinite(got["dx"][:, :100]).all() and torch.isfinite(got["dh0"]).all()
    else:
        assert not torch.isfinite(got["dh0"]).any()


@pytest.mark.parametrize("kind", TYPES)
def test_finite_values_do_not_depend_on_the_array_of_resets(kind):
    """Decays of every strength: with an array without a reset the same bits as without one."""
    t = make(3, 500, 48, kind, h0=True, seed=5, rates=(1e-3, 300.0))
    without = run(t)
    t["reset"] = torch.zeros(3, 500, dtype=torch.uint8, device="cuda")
    assert same(run(t), without)
