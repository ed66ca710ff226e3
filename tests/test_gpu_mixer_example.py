"""The mixer example: streaming equals one call, its gradients match the
float64 reference of the same composition, training lowers the loss."""
import os
import sys

import numpy as np
import pytest
import torch

import _mixer_ref as ref
from _parity import check

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def test_streaming_equals_one_call():
    import delta_mixer
    # o is rounded to bf16 on both ways, 2^-8 each, of sums that differ in their last bits
    assert delta_mixer.prompt_and_stream() <= 2 * 2.0 ** -8


def test_training_lowers_the_loss():
    import delta_mixer
    losses = delta_mixer.train()
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0]


def test_gradients_match_the_reference_composition():
    """Through projection, norm, rotation and delta rule in float64 from the stored bf16 q, k, v.  The chain rounds
    to bf16 six times (qn, kn, do, dq, dk and their gradients): 8 half steps of 2^-8."""
    import delta_mixer
    torch.manual_seed(0)
    m = delta_mixer.DeltaMixer(64, seed=3)
    x = torch.randn(1, 70, 64, device="cuda")
    dy = torch.randn(1, 70, 64, device="cuda")
    _, _, kept = m.forward(x, keep=True)
    got = m.backward(kept, dy)
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v, g, beta = (h(kept[n]) for n in ("q", "k", "v", "g", "beta"))
    pos, freq = kept["pos"].cpu().numpy(), h(m.freq)
    rot = lambda t: ref.turn(ref.norm(t, None, "l2", 1e-6)[0], pos, freq, "half", m.amp)  # noqa: E731
    do = (h(dy) @ h(m.w_out)).reshape(1, 70, m.Hv, m.D)
    scale = m.D ** -0.5
    qn, kn = rot(q), rot(k)
    o, _, _ = ref.delta_forward(qn, kn, v, g, beta, None, scale)
    d = ref.delta_backward(qn, kn, v, g, beta, None, scale, do, None)
    dq, _ = ref.norm_turn_backward(q, None, "l2", 1e-6, pos, freq, "half", m.amp, d["dq"])
    dk, _ = ref.norm_turn_backward(k, None, "l2", 1e-6, pos, freq, "half", m.amp, d["dk"])
    da = -d["dg"] * np.exp(h(m.log_a)) / (1 + np.exp(3.0 - h(kept["a"])))
    db = d["dbeta"] * beta * (1 - beta)
    flat = lambda t: t.reshape(70, -1)  # noqa: E731
    dp = np.concatenate([flat(dq), flat(dk), flat(d["dv"]), flat(da), flat(db)], -1)
    tol = 8 * 2.0 ** -8
    check(h(got["w_in"]), dp.T @ flat(h(x)), tol, "w_in")
    check(h(got["w_out"]), flat(h(dy)).T @ flat(o), tol, "w_out")
    check(h(got["log_a"]), (d["dg"] * g).sum((0, 1)), tol, "log_a")
