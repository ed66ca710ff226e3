"""GPU tests of arrays with more than 2^31 values: the end of a long call against a call on the end alone."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api, init

import _mixer_ref as ref
from test_gpu_delta import BF16, FWD, GRAD

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    yield
    torch.cuda.empty_cache()


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_delta(dt):
    """The state is reset 150 tokens before the end (a chunk's border), so that the tokens after it, their gradients and
    the last state know of nothing before."""
    L, Hk, Hv, D, tail = 64 * 2190 - 42, 8, 128, 128, 150
    assert L * Hv * D > 2 ** 31 and (L - tail) % 64 == 0
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s, t=dt: torch.empty(*s, device="cuda", dtype=t).normal_(generator=gen)  # noqa: E731
    q, k = rnd(1, L, Hk, D), rnd(1, L, Hk, D)
    k /= k.float().norm(dim=-1, keepdim=True).to(dt)
    v, g = rnd(1, L, Hv, D), -rnd(1, L, Hv, t=torch.float32).abs()
    beta, ds = torch.sigmoid(rnd(1, L, Hv, t=torch.float32)), rnd(1, Hv, D, D, t=torch.float32)
    g[:, L - tail] = -float("inf")
    end = [t[:, L - tail:].contiguous() for t in (q, k, v, g, beta)]
    low = BF16 if dt == torch.bfloat16 else 0
    o, s = api.s5_delta_forward(q, k, v, g, beta, s_last=True)
    o2, s2 = api.s5_delta_forward(*end, s_last=True)
    assert off(o[:, L - tail:], o2) <= 2 * (FWD + low) and off(s, s2) <= 2 * FWD
    del o
    saved, saved2 = api.new_delta_saved(q, v), api.new_delta_saved(end[0], end[2])
    api.s5_delta_forward(q, k, v, g, beta, saved=saved)
    api.s5_delta_forward(*end, saved=saved2)
    a = api.s5_delta_backward(q, k, v, g, beta, v, saved, ds_last=ds)
    b = api.s5_delta_backward(*end, end[2], saved2, ds_last=ds)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert off(a[n][:, L - tail:], b[n]) <= 2 * (GRAD * 4 + (low if n in ("dq", "dk", "dv") else 0)), n
    assert not api.s5_delta_fault()


def test_rotation_and_norm():
    L, H, D, tail = 590_003, 32, 128, 37
    assert L * H * D > 2 ** 31
    x = torch.empty(1, L, H, D, device="cuda", dtype=torch.bfloat16).normal_()
    k = x[:, :, :1].contiguous()
    pos, freq = torch.arange(L, device="cuda")[None], torch.from_numpy(init.rotary_frequencies(D)[0]).cuda()
    w = torch.ones(D, device="cuda")
    vx, p = x[:, -tail:].double().cpu().numpy(), pos[:, -tail:].cpu().numpy()
    turned = lambda t: ref.turn(t, p, freq.cpu().numpy(), "half", 1.0)  # noqa: E731
    tol = 16 * 2.0 ** -24 + BF16
    err = lambda t, want: np.linalg.norm(t[:, -tail:].double().cpu().numpy() - want) / np.linalg.norm(want)  # noqa: E731
    assert err(api.s5_rotary(x, pos, freq), turned(vx)) <= tol
    assert err(api.s5_qk_norm_rotary(x, k, pos, freq)[0], turned(ref.norm(vx, None, "rms", 1e-6)[0])) <= tol
    g = api.s5_qk_norm_rotary_backward(x, k, x, k, pos, freq, q_weight=w, k_weight=w)
    want = ref.norm_turn_backward(vx, None, "rms", 1e-6, p, freq.cpu().numpy(), "half", 1.0, vx)[0]
    assert err(g["dq"], want) <= tol + 16 * 2.0 ** -24
    assert not api.s5_rotary_fault()
