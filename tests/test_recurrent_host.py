"""Host checks of the gated recurrence, the short convolution and layer norm of a sum: refusals, buffer sizes, and the
float64 reference forms against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import _native, api

import _recurrent_ref as ref

INV, UNSUP, OK = 1, 2, 0
P, Q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)   # aligned, never dereferenced on rejection
MIS, ODD = ctypes.c_void_p((1 << 20) + 4), ctypes.c_void_p((1 << 20) + 2)


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


def test_scan_sizes(lib):
    assert lib.s5_gated_scan_saved_size(2, 129, 8) >= 4 * 2 * 3 * 8
    assert lib.s5_gated_scan_saved_size(0, 0, 1) > 0
    for bad in ((-1, 8, 8), (1, -1, 8), (1, 8, 0), (1, (1 << 30) + 1, 8), (1 << 30, 8, 64)):
        assert lib.s5_gated_scan_saved_size(*bad) == 0 and lib.s5_gated_scan_workspace_size(*bad) == 0
    with pytest.raises(api.S5Error):
        api.new_gated_scan_saved(torch.empty(1, 8, 0))


def test_scan_forward_refusals(lib):
    n = lib.s5_gated_scan_saved_size(2, 70, 8)
    base = [P, 8, P, 8, P, 8, 0, P, None, None, None, 1, 2, 70, 8, Q, 8, None, None, 0, None]
    fwd = lambda **kw: lib.s5_gated_scan_forward(*_with(base, **kw))  # noqa: E731
    for bad in (dict(_0=None), dict(_0=MIS), dict(_1=7), dict(_2=None), dict(_3=7), dict(_4=MIS), dict(_5=7), dict(_6=2), dict(_7=None),
                dict(_7=MIS), dict(_8=MIS), dict(_10=ODD), dict(_12=-1), dict(_13=-1), dict(_14=0), dict(_15=None), dict(_15=MIS),
                dict(_16=7), dict(_17=MIS), dict(_18=P, _19=n - 1), dict(_18=MIS, _19=n)):
        assert fwd(**bad) == INV, bad
    for bad in (dict(_12=1 << 30, _14=64), dict(_13=(1 << 30) + 1)):
        assert fwd(**bad) == UNSUP, bad
    assert fwd(_12=0) == OK and fwd(_13=0) == OK          # nothing to do without a last state


def test_scan_backward_refusals(lib):
    n, m = lib.s5_gated_scan_saved_size(2, 70, 8), lib.s5_gated_scan_workspace_size(2, 70, 8)
    base = [P, 8, P, 8, P, 8, 0, P, None, None, 1, 2, 70, 8, P, 8, None, P, n, Q, 8, Q, 8, Q, 8, Q, None, P, m, None]
    bwd = lambda **kw: lib.s5_gated_scan_backward(*_with(base, **kw))  # noqa: E731
    for bad in (dict(_0=None), dict(_3=7), dict(_5=7), dict(_6=9), dict(_7=None), dict(_9=ODD), dict(_14=None), dict(_15=7), dict(_16=MIS),
                dict(_17=None), dict(_18=n - 1), dict(_19=None), dict(_20=7), dict(_21=MIS), dict(_22=7), dict(_23=None), dict(_24=7),
                dict(_25=None), dict(_25=MIS), dict(_26=MIS), dict(_27=None), dict(_28=m - 1), dict(_11=-1), dict(_13=0)):
        assert bwd(**bad) == INV, bad
    assert bwd(_12=(1 << 30) + 1) == UNSUP


def test_scan_step_refusals(lib):
    base = [P, P, P, 0, P, 1, 2, 8, P, Q, None]
    for bad in (dict(_0=None), dict(_1=None), dict(_2=MIS), dict(_3=5), dict(_4=None), dict(_6=-1), dict(_7=0), dict(_8=MIS), dict(_9=None)):
        assert lib.s5_gated_scan_step(*_with(base, **bad)) == INV, bad
    assert lib.s5_gated_scan_step(*_with(base, _6=0)) == OK


def test_conv_refusals(lib):
    base = [P, 8, 0, P, None, 0, None, None, None, 2, 9, 8, 4, Q, 8, None, None]
    fwd = lambda **kw: lib.s5_short_conv_forward(*_with(base, **kw))  # noqa: E731
    for bad in (dict(_0=None), dict(_0=MIS), dict(_1=7), dict(_2=2), dict(_3=None), dict(_3=MIS), dict(_4=MIS), dict(_5=2), dict(_6=MIS),
                dict(_8=ODD), dict(_9=-1), dict(_10=-1), dict(_11=0), dict(_12=0), dict(_13=None), dict(_13=P), dict(_14=7), dict(_15=MIS)):
        assert fwd(**bad) == INV, bad
    for bad in (dict(_12=1), dict(_12=9), dict(_10=(1 << 30) + 1), dict(_9=1 << 30)):
        assert fwd(**bad) == UNSUP, bad
    assert fwd(_9=0) == OK and fwd(_10=0) == OK
    m = lib.s5_short_conv_workspace_size(8, 4)
    base = [P, 8, 0, P, P, 1, None, None, None, 2, 9, 8, 4, P, 8, None, Q, 8, Q, Q, None, P, m, None]
    for bad in (dict(_0=None), dict(_13=None), dict(_14=7), dict(_15=MIS), dict(_16=None), dict(_16=P), dict(_17=7), dict(_18=None),
                dict(_19=MIS), dict(_20=MIS), dict(_21=None), dict(_22=m - 1), dict(_5=7)):
        assert lib.s5_short_conv_backward(*_with(base, **bad)) == INV, bad
    assert lib.s5_short_conv_backward(*_with(base, _12=9)) == UNSUP
    assert lib.s5_short_conv_workspace_size(0, 4) == 0 and lib.s5_short_conv_workspace_size(8, 9) == 0
    base = [P, 0, P, None, 1, 2, 8, 4, Q, Q, None]
    for bad in (dict(_0=None), dict(_1=3), dict(_2=None), dict(_3=MIS), dict(_4=5), dict(_5=-1), dict(_8=None), dict(_9=MIS)):
        assert lib.s5_short_conv_step(*_with(base, **bad)) == INV, bad
    assert lib.s5_short_conv_step(*_with(base, _7=9)) == UNSUP
    assert lib.s5_short_conv_step(*_with(base, _5=0)) == OK


def test_norm_refusals(lib):
    base = [P, 8, P, 8, 0, P, P, 1e-5, 5, 8, Q, 8, P, 8, P, None]
    fwd = lambda **kw: lib.s5_add_layernorm(*_with(base, **kw))  # noqa: E731
    for bad in (dict(_0=None), dict(_0=MIS), dict(_1=7), dict(_2=MIS), dict(_3=7), dict(_4=2), dict(_5=MIS), dict(_6=MIS), dict(_7=-1.0),
                dict(_7=float("nan")), dict(_8=-1), dict(_9=0), dict(_10=None), dict(_10=P), dict(_11=7), dict(_12=MIS), dict(_13=7),
                dict(_13=16), dict(_14=MIS)):                # _10: y is total; _13=16: in place with another pitch
        assert fwd(**bad) == INV, bad
    for bad in (dict(_9=16385, _1=16385), dict(_8=1 << 31)):
        assert fwd(**bad) == UNSUP, bad
    assert fwd(_8=0) == OK
    m = lib.s5_add_layernorm_workspace_size(8)
    base = [P, 8, P, 8, P, 8, P, 8, 0, P, P, 5, 8, Q, 8, Q, Q, P, m, None]
    for bad in (dict(_0=None), dict(_1=7), dict(_2=MIS), dict(_3=7), dict(_4=None), dict(_5=7), dict(_6=MIS), dict(_7=7), dict(_8=2),
                dict(_9=MIS), dict(_10=None), dict(_13=None), dict(_14=7), dict(_13=P, _14=16), dict(_15=MIS), dict(_16=MIS), dict(_17=None),
                dict(_18=m - 1)):
        assert lib.s5_add_layernorm_backward(*_with(base, **bad)) == INV, bad
    assert lib.s5_add_layernorm_workspace_size(0) == 0 and lib.s5_add_layernorm_workspace_size(16385) == 0


def test_python_calls_refuse_what_they_cannot_take(lib):
    t = torch.empty(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.s5_gated_scan_forward(t, t, None, t)
    with pytest.raises(ValueError, match="3 axes"):
        api.s5_gated_scan_forward(t[0], t[0], None, t)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.s5_gated_scan_step(t[0].half(), t[0], None, t, t)
    with pytest.raises(ValueError, match="taps"):
        api.s5_short_conv_forward(t, torch.empty(7, 4))
    with pytest.raises(KeyError):
        api.s5_short_conv_forward(t, torch.empty(8, 4), activation="relu")
    with pytest.raises(ValueError, match="without a residual"):
        api.s5_add_layernorm(t, total=t)
    with pytest.raises(api.S5Error):
        api.new_gated_scan_saved(torch.empty(2, 4, 0))


def test_native_half_leaves_the_rest_to_python(lib):
    m, t = _native.marshal(), torch.zeros(2, 3, 8)
    assert m.gated_scan_forward(t, t, None, t, None, None, None, None, True, None, None) is None
    assert m.gated_scan_backward(t, t, None, t, t, t, None, None, None, None, True, None) is None
    assert m.gated_scan_step(t, t, None, t, t, True, None) is None
    assert m.short_conv_forward(t, t, None, 0, None, None, None, None, None) is None
    assert m.short_conv_backward(t, t, t, None, 0, None, None, None, None, None) is None
    assert m.short_conv_step(t, t, t, None, 0, None) is None
    assert m.add_layernorm(t, None, None, None, 1e-5, None, None, None) is None
    assert m.add_layernorm_backward(t, t, t, None, None, None, None, None) is None
    for fn in (m.gated_scan_forward, m.gated_scan_backward, m.gated_scan_step, m.short_conv_forward, m.short_conv_backward,
               m.short_conv_step, m.add_layernorm, m.add_layernorm_backward):
        with pytest.raises(TypeError, match="arguments"):
            fn(t)


RESET = np.array([[0, 0, 1, 0, 0, 0], [1, 0, 0, 0, 1, 1]], bool)
LENGTHS = np.array([4, 6])


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("reset,lengths,normalize", [(None, None, True), (RESET, None, True), (RESET, LENGTHS, False), (None, LENGTHS, True)])
def test_reference_scan_gradients_match_differences(gated, reset, lengths, normalize):
    rng = np.random.default_rng(1)
    B, L, C = 2, 6, 2
    x = dict(x=rng.standard_normal((B, L, C)), ga=rng.standard_normal((B, L, C)), rate=0.1 + rng.random(C), h0=rng.standard_normal((B, C)))
    if gated:
        x["gx"] = rng.standard_normal((B, L, C))
    dh, dl = rng.standard_normal((B, L, C)), rng.standard_normal((B, C))
    kw = dict(reset=reset, lengths=lengths, normalize=normalize)

    def loss(x, ga, rate, h0, gx=None):
        o = ref.scan(x, ga, gx, rate, h0, **kw)
        return (o["h"][0] * dh).sum() + (o["h_last"][0] * dl).sum()

    got = ref.scan(x["x"], x["ga"], x.get("gx"), x["rate"], x["h0"], dh=dh, dh_last=dl, **kw)
    for name, d in ref.differences(loss, x).items():
        key = dict(ga="dgate_a", gx="dgate_x").get(name, "d" + name)
        assert np.allclose(got[key][0], d, rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("reset,lengths", [(None, None), (RESET, None), (RESET, LENGTHS), (None, np.array([0, 2]))])
def test_reference_conv_gradients_match_differences(K, silu, reset, lengths):
    rng = np.random.default_rng(2)
    B, L, C = 2, 6, 2
    x = dict(x=rng.standard_normal((B, L, C)), w=rng.standard_normal((C, K)), bias=rng.standard_normal(C), past=rng.standard_normal((B, K - 1, C)))
    dy, dl = rng.standard_normal((B, L, C)), rng.standard_normal((B, K - 1, C))

    def loss(x, w, bias, past):
        o = ref.conv(x, w, bias, silu, past, reset, lengths)
        return (o["y"][0] * dy).sum() + (o["past_out"][0] * dl).sum()

    got = ref.conv(x["x"], x["w"], x["bias"], silu, x["past"], reset, lengths, dy, dl)
    for name, d in ref.differences(loss, x).items():
        assert np.allclose(got["dweight" if name == "w" else "d" + name][0], d, rtol=1e-6, atol=1e-7), name


def test_reference_conv_parts_are_the_whole():
    """Two calls, the first's past handed on, are one call."""
    rng = np.random.default_rng(3)
    x, w, past = rng.standard_normal((2, 9, 3)), rng.standard_normal((3, 4)), rng.standard_normal((2, 3, 3))
    reset = rng.random((2, 9)) < 0.3
    for cut in range(1, 9):
        a = ref.conv(x[:, :cut], w, None, True, past, reset[:, :cut])
        b = ref.conv(x[:, cut:], w, None, True, a["past_out"][0], reset[:, cut:])
        whole = ref.conv(x, w, None, True, past, reset)
        assert np.allclose(np.concatenate([a["y"][0], b["y"][0]], 1), whole["y"][0])
        assert np.array_equal(b["past_out"][0], whole["past_out"][0])


def test_reference_norm_gradients_match_differences():
    rng = np.random.default_rng(4)
    x = dict(x=rng.standard_normal((3, 5)), weight=rng.standard_normal(5), bias=rng.standard_normal(5), residual=rng.standard_normal((3, 5)))
    dy, dt = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss(**x):
        o = ref.norm(x["x"], x["weight"], x["bias"], x["residual"], 1e-3)
        return (o["y"][0] * dy).sum() + (o["total"][0] * dt).sum()

    o = ref.norm(x["x"], x["weight"], x["bias"], x["residual"], 1e-3)
    got = ref.norm_backward(o["total"][0], dy, o["mean"][0], o["inv"][0], x["weight"], dt)
    for name, d in ref.differences(loss, x).items():
        key = dict(x="dx", residual="dx", weight="dweight", bias="dbias")[name]
        assert np.allclose(got[key][0], d, rtol=1e-6, atol=1e-7), name
