"""GPU tests of the decay's gradient where gates are all but shut: it has to keep its own digits, however small it is
beside the gradients of its neighbours.

Tolerance: 256 half steps of 2^-24 as in test_gpu_delta.py (rel-L2), but over the tokens of one decay at a time."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api

import _mixer_ref as ref
from test_gpu_delta import DG, grads, host, make

pytestmark = pytest.mark.gpu
DECAYS = [0.0, -1e-3, -0.1, -1.0, -3.0, -6.0, -9.0, -12.0, -20.0, -40.0, -80.0]


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def want(v):
    return ref.delta_backward(v["q"], v["k"], v["v"], v["g"], v["beta"], v["s0"], 0.3, v["do"], v["ds_last"])["dg"]


def close_by_decay(got, exact, g):
    got = host(got)
    for x in np.unique(g):
        at = g == x
        off = np.linalg.norm(got[at] - exact[at]) / np.linalg.norm(exact[at])
        print("decay %g: %.2e" % (x, off))
        assert off <= DG, (x, off)


SHAPES = [(1, 150, 1, 11, 128, 128, torch.bfloat16), (2, 100, 1, 11, 64, 128, torch.bfloat16), (1, 64, 11, 22, 128, 64, torch.bfloat16),
          (1, 130, 1, 11, 64, 64, torch.bfloat16), (1, 150, 1, 11, 48, 80, torch.bfloat16), (1, 150, 1, 11, 64, 64, torch.float32),
          (1, 90, 1, 11, 132, 20, torch.float32), (1, 65, 1, 11, 36, 256, torch.float32)]


def set_gates(d, v, g):
    d["g"] = torch.from_numpy(g).float().cuda()
    v["g"] = host(d["g"])


@pytest.mark.parametrize("shape", SHAPES)
def test_heads_of_one_decay(shape):
    """A head for each decay."""
    *sizes, dt = shape
    d, v = make(*sizes, dt=dt, seed=sum(sizes))
    B, L, _, Hv = sizes[:4]
    set_gates(d, v, np.broadcast_to(np.array(DECAYS * (Hv // 11)), (B, L, Hv)).copy())
    close_by_decay(grads(d)["dg"], want(v), v["g"])


@pytest.mark.parametrize("shape", SHAPES)
def test_shut_gates_among_open_ones(shape):
    """Every seventh token has one of the strong decays, the others next to none; some write nothing."""
    *sizes, dt = shape
    d, v = make(*sizes, dt=dt, seed=sum(sizes) + 1)
    B, L, _, Hv = sizes[:4]
    rng = np.random.default_rng(5)
    g = np.full((B, L, Hv), -0.05)
    g[:, ::7] = rng.choice(DECAYS[4:], g[:, ::7].shape)
    set_gates(d, v, g)
    d["beta"][:, ::5] = 0
    v["beta"] = host(d["beta"])
    close_by_decay(grads(d)["dg"], want(v), v["g"])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_gate_that_is_shut_has_no_gradient(dt):
    d, v = make(1, 100, 1, 2, 128, 128, dt=dt, seed=4)
    d["g"][:, 10::9] = -float("inf")
    d["g"][:, 11::9] = -110.0
    dg = grads(d)["dg"]
    assert torch.count_nonzero(dg[:, 10::9]) == 0 and torch.count_nonzero(dg[:, 11::9]) == 0
    assert torch.isfinite(dg).all()
