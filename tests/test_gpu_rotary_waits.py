"""GPU tests of waits that run out inside the streaming rotation: with a limit of
0 ns every copy is given up, still in flight or not.  The kernel ends, stores
nothing of what did not come, and says so; the next call is whole."""
import time

import pytest
import torch

from diagonal_state_space_gb300 import _native, api, init

pytestmark = pytest.mark.gpu
MARK = 7.0


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.fixture
def short():
    lib = _native.lib()
    before = lib.s5_rotary_wait_limit(0)
    yield lib
    lib.s5_rotary_wait_limit(before)
    lib.s5_rotary_fault()


def test_the_limit_is_set_and_given_back():
    lib = _native.lib()
    before = lib.s5_rotary_wait_limit(123)
    assert before == 2_000_000_000 and lib.s5_rotary_wait_limit(before) == 123


# L, heads: two items a warp or one; more items than stages, by token and dealt out
CASES = [(2048, 16, None), (16384, 32, "l2"), (20011, 32, None)]


@pytest.mark.parametrize("L,H,kind", CASES)
def test_a_wait_that_ran_out_ends_the_forward_call(short, L, H, kind):
    lib = short
    x = torch.randn(1, L, H, 128, device="cuda").bfloat16()
    k = x[:, :, :1].contiguous()
    pos, freq = torch.arange(L, device="cuda")[None], torch.from_numpy(init.rotary_frequencies(128)[0]).cuda()

    def call(out):
        if kind is None:
            return api.s5_rotary(x, pos, freq, out=out)
        return api.s5_qk_norm_rotary(x, k, pos, freq, norm=kind, q_out=out)[0]

    lib.s5_rotary_fault()
    got = torch.full_like(x, MARK)
    t0 = time.monotonic()
    call(got)
    assert lib.s5_rotary_fault() == 1 and time.monotonic() - t0 < 1.5
    assert lib.s5_rotary_fault() == 0                       # cleared
    lib.s5_rotary_wait_limit(2_000_000_000)
    want = call(torch.empty_like(x))
    assert lib.s5_rotary_fault() == 0
    # a head is either as it was or right: nothing that had not come was turned and stored
    rows, ref = got[0].flatten(0, 1), want[0].flatten(0, 1)
    untouched, right = (rows == MARK).all(-1), (rows == ref).all(-1)
    assert bool((untouched | right).all()) and bool(untouched.any())


def test_in_place_input_survives_a_wait_that_ran_out(short):
    x = torch.randn(1, 4096, 16, 128, device="cuda").bfloat16()
    before = x.clone()
    pos, freq = torch.arange(4096, device="cuda")[None] + 1, torch.from_numpy(init.rotary_frequencies(128)[0]).cuda()
    api.s5_rotary(x, pos, freq, out=x)
    assert short.s5_rotary_fault() == 1
    short.s5_rotary_wait_limit(2_000_000_000)
    want = api.s5_rotary(before, pos, freq)
    same, right = (x == before).all(-1), (x == want).all(-1)
    assert bool((same | right).all()) and bool(same.any())


@pytest.mark.parametrize("weighted", [True, False])
def test_a_wait_that_ran_out_ends_the_backward_call(short, weighted):
    B, L, H, D = 1, 8192, 16, 128
    q, k, gq, gk = (torch.randn(B, L, H, D, device="cuda").bfloat16() for _ in range(4))
    w = torch.rand(D, device="cuda") + 0.5 if weighted else None
    pos, freq = torch.arange(L, device="cuda")[None], torch.from_numpy(init.rotary_frequencies(D)[0]).cuda()
    api.s5_qk_norm_rotary_backward(q, k, gq, gk, pos, freq, q_weight=w, k_weight=w)
    assert short.s5_rotary_fault() == 1
    short.s5_rotary_wait_limit(2_000_000_000)
    a = api.s5_qk_norm_rotary_backward(q, k, gq, gk, pos, freq, q_weight=w, k_weight=w)
    b = api.s5_qk_norm_rotary_backward(q, k, gq, gk, pos, freq, q_weight=w, k_weight=w)
    assert short.s5_rotary_fault() == 0
    for n in a:
        assert a[n] is b[n] is None or (torch.isfinite(a[n]).all() and torch.equal(a[n], b[n])), n
