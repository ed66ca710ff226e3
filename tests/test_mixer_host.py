"""Host checks of the gated delta rule and rotation calls: refusals, buffer
sizes, frequency tables, and the float64 reference forms against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import _native, api, init

import _mixer_ref as ref

INV, UNSUP, OK = 1, 2, 0
P = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced on rejection
MIS = ctypes.c_void_p((1 << 20) + 4)
ODD = ctypes.c_void_p((1 << 20) + 2)    # not even a float's


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        from diagonal_state_space_gb300 import build
        build.build()
    return _native.lib()


def _with(args, **kw):
    a = list(args)
    for i, v in kw.items():
        a[int(i[1:])] = v
    return a


def test_delta_sizes(lib):
    assert lib.s5_delta_saved_size(0, 0, 1, 4, 4) >= 256
    for bad in ((-1, 8, 2, 8, 8), (1, -1, 2, 8, 8), (1, 8, 0, 8, 8), (1, 8, 2, 6, 8), (1, 8, 2, 8, 260), (1, 8, 2, 0, 8)):
        assert lib.s5_delta_saved_size(*bad) == 0
        assert lib.s5_delta_workspace_size(*bad, 1) == 0
    assert lib.s5_delta_saved_size(2, 128, 4, 8, 16) >= 4 * (2 * 2 * 128 * 4 * 16 + 2 * 4 * 3 * 8 * 16)
    assert lib.s5_delta_workspace_size(2, 128, 4, 8, 16, 1) > lib.s5_delta_workspace_size(2, 128, 4, 8, 16, 0)
    with pytest.raises(api.S5Error, match="multiples of 4"):
        api.new_delta_saved(torch.empty(1, 8, 2, 6), torch.empty(1, 8, 2, 6))


def _fwd(lib, **kw):
    n = lib.s5_delta_workspace_size(2, 8, 4, 8, 8, 0)
    base = [P, 16, P, 16, P, 32, 0, P, P, None, 1.0, 2, 8, 2, 4, 8, 8, P, 32, None, None, 0, P, n, None]
    return lib.s5_delta_forward(*_with(base, **kw))


def test_delta_forward_refusals(lib):
    for bad in (dict(_0=None), dict(_2=MIS), dict(_4=None), dict(_7=None), dict(_8=ODD), dict(_17=None), dict(_9=MIS),
                dict(_19=MIS), dict(_6=7), dict(_1=15), dict(_3=8), dict(_5=31), dict(_18=31), dict(_11=-1), dict(_12=-1),
                dict(_13=3), dict(_13=0), dict(_15=0), dict(_22=None), dict(_23=16), dict(_20=P, _21=16),
                dict(_10=float("nan"))):
        assert _fwd(lib, **bad) == INV, bad
    for bad in (dict(_15=6), dict(_16=260), dict(_11=70000), dict(_12=1 << 30, _11=4)):
        assert _fwd(lib, **bad) == UNSUP, bad
    assert _fwd(lib, _11=0) == OK        # no sequences: nothing is launched


def _bwd(lib, **kw):
    n, m = lib.s5_delta_workspace_size(2, 8, 4, 8, 8, 1), lib.s5_delta_saved_size(2, 8, 4, 8, 8)
    base = [P, 16, P, 16, P, 32, 0, P, P, None, 1.0, 2, 8, 2, 4, 8, 8, P, 32, None, P, m, P, 16, P, 16, P, 32, P, P, None,
            P, n, None]
    return lib.s5_delta_backward(*_with(base, **kw))


def test_delta_backward_refusals(lib):
    for bad in (dict(_0=None), dict(_17=None), dict(_18=31), dict(_20=None), dict(_21=16), dict(_22=None), dict(_23=15),
                dict(_25=15), dict(_27=31), dict(_28=None), dict(_29=MIS), dict(_30=MIS), dict(_31=None), dict(_32=16),
                dict(_19=MIS), dict(_6=2)):
        assert _bwd(lib, **bad) == INV, bad
    assert _bwd(lib, _16=6) == UNSUP
    assert _bwd(lib, _11=0) == OK


def test_delta_step_refusals(lib):
    base = [P, P, P, 0, P, P, 1.0, 2, 2, 4, 8, 8, P, P, None]
    for bad in (dict(_0=None), dict(_1=MIS), dict(_4=None), dict(_5=None), dict(_12=None), dict(_13=MIS), dict(_3=9),
                dict(_7=-1), dict(_8=3), dict(_6=float("nan"))):
        assert lib.s5_delta_step(*_with(base, **bad)) == INV, bad
    for bad in (dict(_10=6), dict(_11=300)):
        assert lib.s5_delta_step(*_with(base, **bad)) == UNSUP, bad
    assert lib.s5_delta_step(*_with(base, _7=0)) == OK


def test_rotary_refusals(lib):
    base = [P, 32, 0, P, P, 8, 0, 1.0, 0, 5, 4, 8, P, 32, None]
    for bad in (dict(_0=None), dict(_0=MIS), dict(_1=31), dict(_2=5), dict(_3=None), dict(_4=None), dict(_5=7), dict(_5=10),
                dict(_5=-2), dict(_6=2), dict(_7=0.0), dict(_7=float("nan")), dict(_9=-1), dict(_12=None), dict(_13=31),
                dict(_13=40)):                       # the last: in place with another pitch
        assert lib.s5_rotary(*_with(base, **bad)) == INV, bad
    for bad in (dict(_11=9, _5=8), dict(_11=258), dict(_9=1 << 31)):
        assert lib.s5_rotary(*_with(base, **bad)) == UNSUP, bad
    assert lib.s5_rotary(*_with(base, _9=0)) == OK
    assert lib.s5_rotary(*_with(base, _10=0)) == OK


def test_qk_norm_rotary_refusals(lib):
    base = [P, 32, P, 16, 0, None, None, 1, 1e-6, P, P, 8, 0, 1.0, 5, 4, 2, 8, P, 32, P, 16, None]
    for bad in (dict(_0=None), dict(_2=None), dict(_5=MIS), dict(_7=3), dict(_8=-1.0), dict(_8=float("nan")), dict(_15=-1),
                dict(_18=None), dict(_19=31), dict(_3=15), dict(_21=40), dict(_12=7)):
        assert lib.s5_qk_norm_rotary(*_with(base, **bad)) == INV, bad
    assert lib.s5_qk_norm_rotary(*_with(base, _17=7, _11=6)) == UNSUP
    assert lib.s5_qk_norm_rotary(*_with(base, _14=0)) == OK
    assert lib.s5_qk_norm_rotary_workspace_size(0) == 0 and lib.s5_qk_norm_rotary_workspace_size(128) > 0
    n = lib.s5_qk_norm_rotary_workspace_size(8)
    base = [P, 32, P, 16, 0, P, P, 1, 1e-6, P, P, 8, 0, 1.0, 5, 4, 2, 8, P, 32, P, 16, P, 32, P, 16, P, P, P, n, None]
    for bad in (dict(_18=None), dict(_22=None), dict(_5=None), dict(_26=MIS), dict(_28=None), dict(_29=16), dict(_23=31),
                dict(_25=40)):
        assert lib.s5_qk_norm_rotary_backward(*_with(base, **bad)) == INV, bad


def test_python_calls_refuse_host_tensors_and_wrong_shapes():
    t = torch.empty(1, 4, 2, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.s5_rotary(t, torch.arange(4)[None], torch.ones(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.s5_delta_step(t[0].half(), t[0].half(), t[0].half(), None, None, None)
    with pytest.raises(ValueError, match="axes"):
        api.s5_delta_step(t, t, t, None, None, None)
    with pytest.raises(ValueError, match="different tokens"):
        api.s5_delta_forward(t, t, torch.empty(1, 5, 2, 8), None, None)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "by_parts"])
def test_rotary_frequencies(scaling):
    f0, _ = init.rotary_frequencies(64)
    f, amp = init.rotary_frequencies(64, scaling=scaling, factor=4.0, trained=4096)
    assert f.dtype == np.float64 and f.shape == (32,)
    assert f0[0] == 1.0 and abs(f0[1] - 10000.0 ** (-1 / 32)) < 1e-15
    if scaling == "none":
        assert np.array_equal(f, f0) and amp == 1.0
    if scaling == "linear":
        assert np.allclose(f, f0 / 4, rtol=1e-15) and amp == 1.0
    if scaling == "ntk":      # the ends of the range: unchanged and divided by the factor
        assert f[0] == 1.0 and abs(f[-1] / (f0[-1] / 4) - 1) < 1e-12 and amp == 1.0
    if scaling == "by_parts":
        turns = 4096 * f0 / (2 * np.pi)
        assert np.array_equal(f[turns >= 32], f0[turns >= 32])
        assert np.allclose(f[turns <= 1], f0[turns <= 1] / 4, rtol=1e-15)
        mid = (turns > 1) & (turns < 32)
        assert mid.any() and np.all((f[mid] < f0[mid]) & (f[mid] > f0[mid] / 4))
        assert abs(amp - (0.1 * np.log(4.0) + 1)) < 1e-15
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, base=-1.0), dict(rot=8, scaling="x"),
                dict(rot=8, scaling="by_parts")):
        with pytest.raises(ValueError):
            init.rotary_frequencies(**bad)


def test_reference_delta_gradients_match_central_differences():
    rng = np.random.default_rng(3)
    B, L, Hk, Hv, Dk, Dv = 1, 5, 1, 2, 3, 2
    x = dict(q=rng.standard_normal((B, L, Hk, Dk)), k=rng.standard_normal((B, L, Hk, Dk)),
             v=rng.standard_normal((B, L, Hv, Dv)), g=-rng.random((B, L, Hv)), beta=rng.random((B, L, Hv)),
             s0=rng.standard_normal((B, Hv, Dk, Dv)))
    do, ds = rng.standard_normal((B, L, Hv, Dv)), rng.standard_normal((B, Hv, Dk, Dv))

    def loss(**y):
        o, s, _ = ref.delta_forward(y["q"], y["k"], y["v"], y["g"], y["beta"], y["s0"], 0.7)
        return (o * do).sum() + (s * ds).sum()

    got = ref.delta_backward(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], 0.7, do, ds)
    for name in x:
        want = np.zeros(x[name].shape)
        for i in np.ndindex(*x[name].shape):
            up, dn = dict(x, **{name: x[name].copy()}), dict(x, **{name: x[name].copy()})
            up[name][i] += 1e-6
            dn[name][i] -= 1e-6
            want[i] = (loss(**up) - loss(**dn)) / 2e-6
        assert np.allclose(got["d" + name], want, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("kind", [None, "rms", "l2"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_norm_and_rotation_gradients_match_central_differences(kind, layout):
    rng = np.random.default_rng(4)
    x, w, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    pos, freq = np.array([0, 7, 100]), np.array([1.0, 0.3])

    def loss(x, w):
        return (ref.turn(ref.norm(x, w, kind, 1e-3)[0], pos, freq, layout, 1.2) * dy).sum()

    dx, dw = ref.norm_turn_backward(x, w, kind, 1e-3, pos, freq, layout, 1.2, dy)
    for i in np.ndindex(*x.shape):
        d = np.zeros(x.shape)
        d[i] = 1e-6
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-6 - dx[i]) < 1e-7
    for i in range(8):
        d = np.zeros(8)
        d[i] = 1e-6
        assert abs((loss(x, w + d) - loss(x, w - d)) / 2e-6 - dw[i]) < 1e-7


def test_native_half_leaves_the_rest_to_python(lib):
    m = _native.marshal()
    q, v, g = torch.zeros(2, 1, 8), torch.zeros(2, 2, 8), torch.zeros(2, 2)
    state = torch.zeros(2, 2, 8, 8)
    assert m.delta_step(q, q, v, g, g, state, None, None) is None           # not on a GPU
    assert m.delta_step(None, q, v, g, g, state, None, None) is None
    assert m.rotary(q, None, None, 0, 1.0, 0, None) is None
    assert m.qk_norm_rotary(q, q, None, None, 1, 1e-6, None, None, 0, 1.0, None, None) is None
    for fn in (m.delta_step, m.delta_forward, m.delta_backward, m.rotary, m.qk_norm_rotary, m.qk_norm_rotary_backward):
        with pytest.raises(TypeError, match="arguments"):
            fn(q)
