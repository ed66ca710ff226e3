"""GPU tests of how many bits the delta rule's bf16 outputs carry before their one rounding, on the tensor cores."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api

import _mixer_ref as ref
from test_gpu_delta import make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def call(d, **kw):
    return api.s5_delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.3, s0=d["s0"], s_last=True, **kw)


@pytest.mark.parametrize("shape", [(10, 200, 8, 8, 128, 64), (13, 130, 4, 8, 64, 64)])
def test_o_does_not_depend_on_what_is_kept(shape):
    """Heads of this number and size take the same slices with and without `saved`: the same sums in the same order."""
    d, _ = make(*shape, dt=torch.bfloat16, seed=3)
    o, s = call(d)
    o2, s2 = call(d, saved=api.new_delta_saved(d["q"], d["v"]))
    assert torch.equal(s, s2) and torch.equal(o, o2)


def rounded(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("shape", [(1, 1024, 2, 4, 128, 128), (3, 300, 16, 32, 128, 128), (2, 400, 20, 20, 64, 64)])
@pytest.mark.parametrize("keep", [False, True])
def test_o_is_rounded_once(shape, keep):
    """o before its rounding is off by at most 32 half steps of 2^-24 (rel-L2).  A value that lies within an error e of
    the border between two bf16 values may take the wrong one: chance 2 e / step, cost step^2, step at most 2^-7 of the
    value.  So the square of the rel-L2 distance from the rounded exact o is at most 2 * 32 * 2^-24 * 2^-7 = 2^-25."""
    d, v = make(*shape, dt=torch.bfloat16, seed=5)
    o = call(d, saved=api.new_delta_saved(d["q"], d["v"]) if keep else None)[0]
    want = rounded(ref.delta_forward(v["q"], v["k"], v["v"], v["g"], v["beta"], v["s0"], 0.3)[0])
    off = np.linalg.norm(o.double().cpu().numpy() - want) / np.linalg.norm(want)
    print("off", off)
    assert off <= 2.0 ** -12.5, off
