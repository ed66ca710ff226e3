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


def dk_reference(x, scale):
    """dk of sequences without an initial state and with no gradient of o, token by token in float64 on the GPU."""
    k, v, g, beta, z = (x[n].double() for n in ("k", "v", "g", "beta", "ds_last"))
    s, faded, e = torch.zeros_like(z), [], []
    for t in range(k.shape[1]):
        f = torch.exp(g[:, t])[..., None, None] * s
        faded.append(f)
        e.append(v[:, t] - torch.einsum("bhkv,bhk->bhv", f, k[:, t]))
        s = f + k[:, t, :, :, None] * (beta[:, t, :, None] * e[t])[:, :, None]
    dk = torch.zeros_like(k)
    for t in reversed(range(k.shape[1])):
        dv = beta[:, t, :, None] * torch.einsum("bhkv,bhk->bhv", z, k[:, t])
        dk[:, t] = torch.einsum("bhkv,bhv->bhk", z, beta[:, t, :, None] * e[t]) - torch.einsum("bhkv,bhv->bhk", faded[t], dv)
        z = torch.exp(g[:, t])[..., None, None] * (z - k[:, t, :, :, None] * dv[:, :, None])
    return dk


def test_dk_is_not_drawn_towards_zero():
    """The adjoint of a chunk's end, and what it is multiplied with, enter dk in two bf16 parts.  Rounded, they are off
    to either side; cut off, by 7e-6 of each value towards zero, and so is the product of second parts left out.  Taken of the difference from the rounded exact dk, since a rounding to bf16 has a
    slope of its own: it is not symmetric at powers of two.  The roundings of 4 million values (2^-8 / sqrt(12) of each)
    would leave 6e-7 in the slope: six times that, 2^-18, is the bound."""
    B, L, H, D = 64, 64, 8, 128
    d, _ = make(B, L, H, H, D, D, dt=torch.bfloat16, s0=False, seed=9)
    gen = torch.Generator(device="cuda").manual_seed(1)
    d["ds_last"] = torch.randn(B, H, D, D, generator=gen, device="cuda")
    d["g"] *= 0.01
    saved = api.new_delta_saved(d["q"], d["v"])
    five = [d[n] for n in ("q", "k", "v", "g", "beta")]
    api.s5_delta_forward(*five, scale=0.3, saved=saved)
    got = api.s5_delta_backward(*five, torch.zeros_like(d["v"]), saved, scale=0.3, ds_last=d["ds_last"])["dk"].double()
    want = dk_reference(d, 0.3)
    slope = float(((got - want.bfloat16().double()) * want).sum() / (want * want).sum())
    print("slope", slope)
    assert abs(slope) <= 2.0 ** -18, slope
