"""GPU tests of the gated delta rule against the float64 recurrence.

Tolerances (rel-L2).  A rounding to fp32 is off by at most 2^-24 of the value,
one to bf16 by 2^-8.  Forward values pass through sums of at most 20 terms in
a row, three per token, whose errors later tokens contract: 32 half steps.  A
gradient goes through the forward values and an adjoint of the same form: 64.
dg adds up to 64 signed terms of its neighbours' size on top: 256.  Outputs in
bf16 get the one rounding of the type besides.
"""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import _native, api

import _mixer_ref as ref
from _parity import check

pytestmark = pytest.mark.gpu

H32 = 2.0 ** -24
FWD, GRAD, DG = 32 * H32, 64 * H32, 256 * H32
BF16 = 2.0 ** -8


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def make(B, L, Hk, Hv, Dk, Dv, dt=torch.float32, s0=True, seed=0, gates="mixed"):
    """Inputs on the GPU and their stored values in float64."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, L, Hk, Dk)) + 0.3
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    x = dict(q=rng.standard_normal((B, L, Hk, Dk)), k=k, v=rng.standard_normal((B, L, Hv, Dv)))
    g = -np.exp(rng.uniform(np.log(1e-4), np.log(3.0), (B, L, Hv)))
    beta = 1 / (1 + np.exp(-2 * rng.standard_normal((B, L, Hv))))
    if gates == "resets":          # states cleared in mid-sequence, by -inf, the lowest value and a large one
        g[rng.random(g.shape) < 0.05] = -np.inf
        g[rng.random(g.shape) < 0.05] = np.finfo(np.float32).min
        g[rng.random(g.shape) < 0.05] = -150.0
        beta[rng.random(beta.shape) < 0.2] = 0.0
    if gates == "none":            # no decay, every key written whole
        g[:], beta[:] = 0.0, 1.0
    if gates == "strong":
        g *= 8
    x.update(g=g, beta=beta, do=rng.standard_normal((B, L, Hv, Dv)))
    x["s0"] = rng.standard_normal((B, Hv, Dk, Dv)) if s0 else None
    x["ds_last"] = rng.standard_normal((B, Hv, Dk, Dv)) if s0 else None
    dev = {n: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(
        dt if n in ("q", "k", "v", "do") else torch.float32) for n, a in x.items()}
    val = {n: None if t is None else t.double().cpu().numpy() for n, t in dev.items()}
    return dev, val


def host(t):
    return t.double().cpu().numpy()


def forward(d, **kw):
    return api.s5_delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.3, s0=d["s0"], s_last=True, **kw)


def expect(v):
    return ref.delta_forward(v["q"], v["k"], v["v"], v["g"], v["beta"], v["s0"], 0.3)[:2]


def close(got, want, tol, what):
    got = host(got) if isinstance(got, torch.Tensor) else got
    want = np.where(np.abs(want) < 2.0 ** -149, 0.0, want)     # exp(-150) is nothing that 32 bits can hold
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what
    if np.linalg.norm(want) == 0:
        assert np.abs(got).max(initial=0.0) == 0, what
    elif want.size:
        check(got, want, tol, what)


SHAPES = [
    (1, 1, 1, 1, 4, 4), (2, 2, 1, 3, 20, 12), (1, 63, 2, 2, 64, 64), (1, 64, 2, 4, 64, 128), (2, 65, 2, 4, 128, 64),
    (1, 200, 1, 2, 128, 128), (2, 130, 2, 2, 48, 80), (1, 70, 1, 1, 256, 256), (1, 129, 1, 2, 132, 260 - 4),
    (1, 1, 2, 4, 128, 128), (3, 17, 2, 6, 128, 128),
]


# As many heads as take wider slices, and two slices a block
MANY = [(3, 130, 8, 16, 128, 128), (5, 100, 8, 16, 128, 128), (11, 70, 4, 8, 64, 64), (10, 129, 4, 8, 64, 128),
        (10, 70, 8, 8, 128, 64)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES + MANY)
def test_forward(shape, dt):
    d, v = make(*shape, dt=dt, seed=sum(shape))
    o, s = forward(d)
    wo, ws = expect(v)
    assert o.dtype == dt and s.dtype == torch.float32
    close(o, wo, FWD + (BF16 if dt == torch.bfloat16 else 0), "o")
    close(s, ws, FWD, "s_last")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates", ["resets", "none", "strong"])
@pytest.mark.parametrize("D", [128, 64, 36])
def test_forward_gates(gates, D, dt):
    d, v = make(2, 150, 1, 2, D, D, dt=dt, gates=gates, seed=7)
    o, s = forward(d)
    wo, ws = expect(v)
    close(o, wo, FWD + (BF16 if dt == torch.bfloat16 else 0), "o")
    close(s, ws, FWD, "s_last")


def test_an_all_reset_sequence_only_sees_its_own_token():
    d, v = make(1, 100, 1, 1, 128, 128, dt=torch.bfloat16, seed=9)
    d["g"].fill_(-float("inf"))
    v["g"][:] = -np.inf
    o, s = forward(d)
    wo, ws = expect(v)
    close(o, wo, FWD + BF16, "o")
    close(s, ws, FWD, "s_last")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_long_sequence(dt):
    d, v = make(1, 4100, 1, 2, 128, 128, dt=dt, seed=11, s0=False)
    o, s = forward(d)
    wo, ws = expect(v)
    close(o, wo, FWD + (BF16 if dt == torch.bfloat16 else 0), "o")
    close(s, ws, FWD, "s_last")


def test_empty_sequence_keeps_the_state():
    d, v = make(2, 0, 1, 2, 64, 64, seed=1)
    o, s = forward(d)
    assert o.shape == (2, 0, 2, 64) and torch.equal(s, d["s0"])
    d["s0"] = None
    assert torch.count_nonzero(forward(d)[1]) == 0
    d, v = make(0, 5, 1, 2, 64, 64, seed=1)
    assert forward(d)[0].shape == (0, 5, 2, 64)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", [0, 3])
def test_slices_of_one_projection(dt, odd):
    """q, k, v as views of one array, whose pitch need not be a multiple of anything."""
    B, L, Hk, Hv, D = 2, 90, 2, 4, 128
    d, v = make(B, L, Hk, Hv, D, D, dt=dt, seed=5)
    base = 16 // dt.itemsize
    fused = torch.full((B, L, 2 * Hk * D + Hv * D + base + odd), float("nan"), device="cuda", dtype=dt)
    views = {}
    at = base
    for n, h in (("q", Hk), ("k", Hk), ("v", Hv)):
        w = fused[:, :, at:at + h * D].unflatten(-1, (h, D))
        w.copy_(d[n])
        views[n] = w
        at += h * D
    o, s = forward(d)
    o2, s2 = forward(dict(d, **views))
    wo, ws = expect(v)
    close(o2, wo, FWD + (BF16 if dt == torch.bfloat16 else 0), "o")
    close(s2, ws, FWD, "s_last")
    if not odd:
        assert torch.equal(o, o2) and torch.equal(s, s2)
    wide = torch.zeros(B, L, Hv * D + 8, device="cuda", dtype=dt)
    out = wide[:, :, :Hv * D].unflatten(-1, (Hv, D))
    api.s5_delta_forward(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.3, s0=d["s0"], o=out)
    assert torch.equal(out, o) and torch.count_nonzero(wide[:, :, Hv * D:]) == 0


def test_refuses_other_strides():
    d, _ = make(2, 8, 2, 2, 64, 64)
    with pytest.raises(ValueError, match="heads must be contiguous"):
        forward(dict(d, q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(ValueError, match="evenly spaced"):
        forward(dict(d, q=torch.zeros(2, 9, 2, 64, device="cuda")[:, :8]))
    with pytest.raises(ValueError, match="shape"):
        forward(dict(d, g=d["g"][:, :4].contiguous()))
    with pytest.raises(ValueError, match="must be torch.float32"):
        forward(dict(d, beta=d["beta"].double()))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_two_calls_equal_one_and_states_may_be_in_place(dt):
    d, v = make(2, 150, 1, 2, 128, 128, dt=dt, seed=21)
    o, s = forward(d)
    cut = lambda a, b: {n: t[:, a:b].contiguous() if n in ("q", "k", "v", "g", "beta") else t for n, t in d.items()}  # noqa: E731
    state = d["s0"].clone()
    parts = []
    for a, b in ((0, 64), (64, 101), (101, 102), (102, 150)):
        c = cut(a, b)
        parts.append(api.s5_delta_forward(c["q"], c["k"], c["v"], c["g"], c["beta"], scale=0.3, s0=state, s_last=state)[0])
    tol = 2 * FWD + (2 * BF16 if dt == torch.bfloat16 else 0)
    close(torch.cat(parts, 1), host(o), tol, "o")
    close(state, host(s), 2 * FWD, "s_last")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 4, 4), (3, 2, 6, 48, 80), (2, 2, 4, 128, 128), (1, 1, 2, 256, 132), (9, 1, 3, 64, 36),
                                   (17, 2, 4, 128, 128), (33, 1, 2, 48, 80), (11, 3, 6, 64, 64), (70, 1, 1, 20, 12),
                                   (64, 1, 1, 128, 68)])
def test_step(shape, dt):
    B, Hk, Hv, Dk, Dv = shape
    d, v = make(B, 6, Hk, Hv, Dk, Dv, dt=dt, seed=31, gates="resets")
    wo, ws = expect(v)
    state = d["s0"].clone()
    for t in range(6):
        o = api.s5_delta_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), state, scale=0.3)
        close(o, wo[:, t], FWD + (BF16 if dt == torch.bfloat16 else 0), "o[%d]" % t)
    close(state, ws, FWD, "state")


def grads(d, **kw):
    saved = api.new_delta_saved(d["q"], d["v"])
    forward(d, saved=saved)
    return api.s5_delta_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], saved, scale=0.3, s0=d["s0"],
                                 ds_last=d["ds_last"], **kw)


def close_grads(got, v, dt):
    want = ref.delta_backward(v["q"], v["k"], v["v"], v["g"], v["beta"], v["s0"], 0.3, v["do"], v["ds_last"])
    low = BF16 if dt == torch.bfloat16 else 0
    for n, w in want.items():
        if n == "ds0" and v["s0"] is None:
            assert got[n] is None
            continue
        tol = DG if n == "dg" else GRAD + (low if n in ("dq", "dk", "dv") else 0)
        close(got[n], w, tol, n)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES + MANY)
def test_backward(shape, dt):
    d, v = make(*shape, dt=dt, seed=sum(shape) + 1)
    close_grads(grads(d), v, dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates", ["resets", "none", "strong"])
@pytest.mark.parametrize("D", [128, 36])
def test_backward_gates(gates, D, dt):
    d, v = make(1, 150, 1, 2, D, D, dt=dt, gates=gates, s0=gates != "strong", seed=8)
    close_grads(grads(d), v, dt)


def test_backward_of_an_empty_sequence():
    d, _ = make(2, 0, 1, 2, 64, 64, seed=1)
    g = grads(d)
    assert torch.equal(g["ds0"], d["ds_last"]) and g["dq"].shape == (2, 0, 1, 64)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_gradients_match_differences_of_the_forward_call(dt):
    """Along one direction per input: (L(x + h d) - L(x - h d)) / 2h in float64 of fp32 outputs.  A difference of
    values of size |L| that carry 32 half steps each is off by 64 * 2^-24 |o| / 2h, the curvature by about h^2."""
    d, v = make(1, 90, 1, 2, 128, 128, seed=41)
    if dt == torch.bfloat16:
        for n in ("q", "k", "v", "do"):
            d[n] = d[n].to(dt)
    g = {n: host(t) for n, t in grads(d).items()}
    f = {n: d[n].float() if d[n].dtype == torch.bfloat16 else d[n] for n in d}
    for n in ("q", "k", "v", "g", "beta", "s0"):
        rng = torch.Generator(device="cuda").manual_seed(2)
        way = torch.randn(f[n].shape, generator=rng, device="cuda")
        way = way / way.norm() * 0.1

        def loss(sign):
            x = dict(f, **{n: f[n] + sign * way})
            o, s = forward(x)
            return float((o.double() * f["do"].double()).sum() + (s.double() * f["ds_last"].double()).sum())

        want = (loss(1) - loss(-1)) / 2
        got = float((g["d" + n] * host(way)).sum())
        size = np.linalg.norm(g["d" + n]) * 0.1
        assert abs(got - want) <= 0.02 * size, (n, got, want, size)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_equal_inputs_give_equal_bits(dt):
    d, _ = make(2, 200, 2, 4, 128, 128, dt=dt, seed=51)
    a, b = grads(d), grads(d)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert all(torch.equal(x, y) for x, y in zip(forward(d), forward(d)))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_other_stream_and_graph(dt):
    d, v = make(2, 140, 1, 2, 128, 128, dt=dt, seed=61)
    want, wg = forward(d), grads(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = forward(d, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gs = forward(d)
        gg = grads(d)
    go.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(go, want[0]) and torch.equal(gs, want[1])
    for n in wg:
        assert torch.equal(gg[n], wg[n]), n


@pytest.mark.parametrize("shape", [(1, 1024, 1, 2, 128, 128), (2, 8200, 2, 4, 64, 128), (3, 2770, 8, 8, 128, 64)])
def test_long_sequences_with_a_state(shape):
    """The preparation of later chunks runs beside the scan of earlier ones: same results in a row, on one workspace
    and in a captured graph."""
    d, v = make(*shape, dt=torch.bfloat16, seed=shape[1])
    wo, ws = expect(v)
    B, L, _, Hv, Dk, Dv = *shape[:3], *shape[3:]
    work = torch.empty(api.s5_delta_workspace_size(B, L, Hv, Dk, Dv), dtype=torch.uint8, device="cuda")
    runs = [forward(d, workspace=work) for _ in range(3)]
    close(runs[0][0], wo, FWD + BF16, "o")
    close(runs[0][1], ws, FWD, "s_last")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        runs += [forward(d, workspace=work) for _ in range(2)]
    for o, s in runs[3:]:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for o, s in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(s, runs[0][1])


def test_nan_stays_in_its_sequence_and_head():
    d, v = make(2, 100, 1, 2, 128, 128, dt=torch.bfloat16, seed=71)
    clean = forward(d)
    d["v"][1, 30, 1, 5] = float("nan")
    d["g"][0, 10, 0] = float("nan")
    o, s = forward(d)
    assert torch.equal(o[0, :, 1], clean[0][0, :, 1]) and torch.equal(o[1, :, 0], clean[0][1, :, 0])
    assert torch.isnan(s[1, 1, :, 5]).any() and torch.isnan(s[0, 0]).all()


def test_no_wait_ran_out():
    d, _ = make(2, 300, 2, 4, 128, 128, dt=torch.bfloat16, seed=81)
    forward(d)
    grads(d)
    assert _native.lib().s5_delta_fault() == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_native_and_python_marshalling_agree(dt):
    d, _ = make(2, 70, 1, 2, 64, 64, dt=dt, seed=91)
    here = torch.cuda.current_stream()
    a, b = forward(d), forward(d, stream=here)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    saved = api.new_delta_saved(d["q"], d["v"])
    forward(d, saved=saved)
    x = [d[n] for n in ("q", "k", "v", "g", "beta", "do")]
    for kw in ({}, dict(s0=d["s0"], ds_last=d["ds_last"])):
        a, b = api.s5_delta_backward(*x, saved, **kw), api.s5_delta_backward(*x, saved, stream=here, **kw)
        assert list(a) == list(b)
        for n in a:
            assert a[n] is b[n] is None or (a[n].dtype is b[n].dtype and torch.equal(a[n], b[n])), n
    tok = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    s1, s2 = d["s0"].clone(), d["s0"].clone()
    assert torch.equal(api.s5_delta_step(*tok, s1), api.s5_delta_step(*tok, s2, stream=here)) and torch.equal(s1, s2)


def test_native_marshalling_refuses_as_python_does():
    d, _ = make(1, 5, 1, 2, 64, 64, seed=92)
    x = [d[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError, match="g must have shape"):
        api.s5_delta_forward(*x[:3], x[3][:, :3].contiguous(), x[4])
    with pytest.raises(ValueError, match="beta must be"):
        api.s5_delta_forward(*x[:4], x[4].double())
    with pytest.raises(api.S5Error):                    # a saved buffer that is too small
        api.s5_delta_forward(*x, saved=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(api.S5Error):
        api.s5_delta_forward(*x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        api.s5_delta_step(*x, d["s0"])
