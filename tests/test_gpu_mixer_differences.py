"""GPU tests of the mixer's gradients against differences of the forward call, along the gradient itself.

Along way = gradient / |gradient| * h the loss rises by |gradient| h, so that a gradient of the other sign, of another
size or of the wrong entries shows at once: the derivative of the loss along any other unit vector u is |gradient| times
the cosine between the two.

Tolerance of (L(+) - L(-)) / 2 over |gradient| h: an output carries 32 half steps of 2^-24 (rel-L2, as in
test_gpu_delta.py), 2^-19, so a loss is off by at most 2^-19 (|do| |o| + |ds| |s|), and this difference by as much; the
third-order term is of the order of h^2 / 6 of the first for steps h relative to the size of what is moved, at most
0.05^2 (rows that do not know of each other are moved by as much each).  Both are worked out below; the sum has to stay under 2 %, or the test says nothing."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api, init

import _mixer_ref as ref
from test_gpu_delta import grads, host, make

pytestmark = pytest.mark.gpu
STEP = 0.05


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def verdicts(want, got, noise):
    """Whether the difference agrees with the gradient, and with spoilt ones: negated, half as much again."""
    tol = noise + STEP * STEP
    assert tol < 0.02, tol
    agrees = lambda g: abs(want / g - 1) <= tol  # noqa: E731
    return agrees(got), agrees(-got), agrees(1.5 * got)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "s0"])
def test_delta(name, dt):
    """Gradients of either path against differences of the fp32 forward call on the same values."""
    d, _ = make(1, 90, 1, 2, 128, 128, seed=41)
    if dt == torch.bfloat16:
        for n in ("q", "k", "v", "do"):
            d[n] = d[n].to(dt)
    g = grads(d)["d" + name].double()
    f = {n: t.float() for n, t in d.items()}
    do, ds = f["do"].double(), f["ds_last"].double()

    def outputs(sign):
        x = dict(f, **{name: (f[name].double() + sign * way).float()})
        return [t.double() for t in api.s5_delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=0.3, s0=x["s0"],
                                                         s_last=True)]

    h = STEP * float(f[name].norm()) / f[name].numel() ** 0.5      # |way|: the size of one value, spread over all
    way = g / g.norm() * h
    (o1, s1), (o0, s0) = outputs(1), outputs(-1)
    want = float(((o1 - o0) * do).sum() + ((s1 - s0) * ds).sum()) / 2
    noise = 2.0 ** -19 * float(do.norm() * o0.norm() + ds.norm() * s0.norm()) / float(g.norm() * h)
    if dt == torch.bfloat16 and name in ("q", "k", "v"):
        noise += 2.0 ** -8                                          # the gradient's own rounding
    assert verdicts(want, float(g.norm()) * h, noise) == (True, False, False)


@pytest.mark.parametrize("kind", ["rms", "l2", None])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("L", [40, 6000])
def test_norm_and_rotation(L, layout, kind):
    """The small and the streaming form; the loss in float64 of the fp32 outputs."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = dict(q=rnd(1, L, 4, 64), k=rnd(1, L, 2, 64), wq=1 + 0.2 * rnd(64), wk=1 + 0.2 * rnd(64))
    dq, dk = rnd(1, L, 4, 64), rnd(1, L, 2, 64)
    pos, freq = torch.arange(L, device="cuda")[None] + 3, torch.from_numpy(init.rotary_frequencies(48)[0]).cuda()
    kw = dict(norm=kind, eps=1e-3, layout=layout, amplitude=1.1)
    g = api.s5_qk_norm_rotary_backward(x["q"], x["k"], dq, dk, pos, freq, q_weight=x["wq"], k_weight=x["wk"], **kw)

    def loss(v):
        a, b = api.s5_qk_norm_rotary(v["q"], v["k"], pos, freq, q_weight=v["wq"], k_weight=v["wk"], **kw)
        return a.double(), b.double()

    for n in x:
        way = g["d" + n].double()
        size = float(way.norm())
        h = STEP * float(x[n].norm()) / x[n].shape[-1] ** 0.5      # a value's size in every row
        way = way / size * h
        (a1, b1), (a0, b0) = (loss(dict(x, **{n: (x[n].double() + s * way).float()})) for s in (1, -1))
        want = float(((a1 - a0) * dq.double()).sum() + ((b1 - b0) * dk.double()).sum()) / 2
        # 16 roundings of 2^-24 an output, those of different rows independent: six deviations of their sum
        noise = 6 / (6 * L) ** 0.5 * 2.0 ** -20 * float(dq.double().norm() * a0.norm() + dk.double().norm() * b0.norm()) / (size * h)
        assert verdicts(want, size * h, noise) == (True, False, False), n


def test_the_reference_passes_and_spoilt_gradients_do_not():
    """The same test of the float64 reference on the CPU: what is wrong by sign, size or place is found."""
    d, v = make(1, 40, 1, 2, 32, 32, seed=3)
    good = ref.delta_backward(v["q"], v["k"], v["v"], v["g"], v["beta"], v["s0"], 0.3, v["do"], v["ds_last"])
    for n in ("q", "k", "v", "g", "beta", "s0"):
        def loss(way):
            y = dict(v, **{n: v[n] + way})
            o, s, _ = ref.delta_forward(y["q"], y["k"], y["v"], y["g"], y["beta"], y["s0"], 0.3)
            return (o * v["do"]).sum() + (s * v["ds_last"]).sum()

        h = STEP * np.linalg.norm(v[n]) / v[n].size ** 0.5
        for spoil, ok in ((lambda a: a, True), (lambda a: -a, False), (lambda a: np.roll(a, 1, -1), False)):
            g = spoil(good["d" + n])
            size = np.linalg.norm(g)
            want = (loss(g / size * h) - loss(-g / size * h)) / 2
            assert verdicts(want, size * h, 1e-9)[0] == ok, n
