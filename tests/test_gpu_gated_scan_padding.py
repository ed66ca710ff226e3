"""GPU tests of what the gated recurrence does not see: padding behind a row's end, a reset's gate, a gradient that a reset
cuts off.  What may hold anything there holds NaN and infinities, and every output is the clean inputs' to the bit."""
import pytest
import torch

from _recurrent_gpu import TYPES, same
from test_gpu_gated_scan import make, run

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def copied(t):
    return {n: a if a is None else a.clone() for n, a in t.items()}


# channels for TMA, pairs and single ones; one tile, and several of a cluster
WIDTHS = [40, 42, 41, 128]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("L,lengths", [(30, [7, 0, 30, 29]), (700, [1, 650, 333, 640])])
@pytest.mark.parametrize("what", [NAN, INF, -INF])
def test_padding_is_not_seen(what, L, lengths, C, gated, kind):
    t = make(4, L, C, kind, gated=gated, h0=True, marks=0.02, seed=L + C)
    t["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    dirty = copied(t)
    for n in ("x", "ga", "dh") + (("gx",) if gated else ()):
        for b, n_b in enumerate(lengths):
            dirty[n][b, n_b:] = what
    for normalize in (True, False):
        got = run(dirty, normalize)
        assert same(got, run(t, normalize))
        for n in ("h", "dx", "dgate_a") + (("dgate_x",) if gated else ()):
            for b, n_b in enumerate(lengths):
                assert torch.count_nonzero(got[n][b, n_b:]) == 0, n


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_padding_is_zeros_whatever_arrives_from_behind(C, kind):
    """A last gradient that is not finite goes through the row, not into its padding."""
    t = make(2, 100, C, kind, h0=True, seed=C)
    t["lengths"] = torch.tensor([60, 0], dtype=torch.int32, device="cuda")
    t["dh_last"][0], t["dh_last"][1] = NAN, INF
    got = run(t)
    for n in ("dx", "dgate_a", "dgate_x"):
        assert torch.count_nonzero(got[n][0, 60:]) == 0 and torch.count_nonzero(got[n][1]) == 0, n
    assert torch.isnan(got["dh0"][0]).all() and torch.isinf(got["dh0"][1]).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("what", [NAN, INF, -INF])
def test_a_resets_gate_is_not_seen(what, C, kind):
    t = make(2, 300, C, kind, h0=True, seed=C)
    t["reset"] = torch.zeros(2, 300, dtype=torch.bool, device="cuda")
    for b, at in ((0, 0), (0, 64), (0, 171), (0, 299), (1, 5), (1, 6)):
        t["reset"][b, at] = True
    dirty = copied(t)
    dirty["ga"][t["reset"]] = what
    got = run(dirty)
    assert same(got, run(t))
    assert torch.count_nonzero(got["dgate_a"][t["reset"]]) == 0


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_a_gradient_ends_at_its_reset(C, kind):
    """NaN that arrives at a reset's token is the input's; the gate and its rate, which the reset does not use, get nothing."""
    t = make(1, 200, C, kind, h0=True, seed=C)
    t["reset"] = torch.zeros(1, 200, dtype=torch.bool, device="cuda")
    t["reset"][0, 90] = True
    dirty = copied(t)
    dirty["dh"][0, 90] = NAN
    clean, got = run(t), run(dirty)
    assert torch.isnan(got["dx"][0, 90]).all() and torch.isnan(got["dgate_x"][0, 90]).all()
    for n in ("dx", "dgate_x"):
        got[n][0, 90] = clean[n][0, 90] = 0
    assert same(got, clean)
