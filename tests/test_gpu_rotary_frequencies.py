"""GPU test of broken frequency tables: what is not finite shows in its pair, and in no other."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api, init

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("L,D,rot", [(5, 128, 64), (5, 18, 6), (5, 20, 20), (12000, 128, 64)])
def test_a_frequency_that_is_not_finite_makes_its_pair_nan(L, D, rot, layout):
    n = rot // 2
    freq = init.rotary_frequencies(rot)[0]
    bad = freq.copy()
    broken = [0, n - 1] if n < 4 else [1, 2, n - 1]
    bad[broken] = [np.nan, -np.inf, np.inf][:len(broken)]
    x = torch.randn(1, L, 3, D, device="cuda")
    pos = torch.arange(L, device="cuda")[None]
    good_t, bad_t = torch.from_numpy(freq).cuda(), torch.from_numpy(bad).cuda()
    mask = torch.zeros(D, dtype=torch.bool, device="cuda")
    for i in broken:
        mask[[i, i + n] if layout == "half" else [2 * i, 2 * i + 1]] = True
    for call in (lambda f: api.s5_rotary(x, pos, f, layout=layout), lambda f: api.s5_rotary(x, pos, f, layout=layout, inverse=True),
                 lambda f: api.s5_qk_norm_rotary(x, x, pos, f, layout=layout)[1]):
        want, got = call(good_t), call(bad_t)
        assert torch.isnan(got[..., mask]).all()
        assert torch.equal(got[..., ~mask], want[..., ~mask])
    g = api.s5_qk_norm_rotary_backward(x, x, x, x, pos, bad_t, norm=None, layout=layout)["dq"]
    assert torch.isnan(g[..., mask]).all() and torch.isfinite(g[..., ~mask]).all()


@pytest.mark.parametrize("start", [1 << 44, 1 << 50, (1 << 52) + 3])
def test_phases_at_far_positions_are_as_good_as_stated(start):
    """|p| max(1, |freq|) 2^-63 turns, and the 16 roundings of 2^-24 of test_gpu_rotary.py; the angles from exact
    integer products.  A pair's values are off by at most its length times the angle's error."""
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    freq = np.array([1.0, 0.37, 1e-3, 3e-5, 7e-9, 30.0, -2.5, 1000.0])
    n, pos = len(freq), torch.arange(6, device="cuda") + start
    x = torch.randn(6, 2, 2 * n, device="cuda")
    vx = x.double().cpu().numpy()
    turns = np.array([[float((Fraction(int(p)) * Fraction(float(f)) / two_pi) % 1) for f in freq] for p in pos.tolist()])
    c = (vx[..., :n] + 1j * vx[..., n:]) * np.exp(2j * np.pi * turns)[:, None, :]
    y = api.s5_rotary(x, pos, torch.from_numpy(freq).cuda()).double().cpu().numpy()
    off = np.abs(y[..., :n] + 1j * y[..., n:] - c) / np.abs(c)
    bound = 2 * np.pi * (start + 6) * np.maximum(1, np.abs(freq)) * 2.0 ** -63 + 16 * 2.0 ** -24
    assert (off <= bound).all(), off.max((0, 1)) / bound
