"""Host checks of which device and stream the recurrent block's calls launch on, with the stand-ins of
test_mixer_devices.py for tensors of several GPUs, for streams and for the library."""
import pytest
import torch

from diagonal_state_space_gb300 import _native, api

from test_mixer_devices import OnGpu, Stream, returned, world  # noqa: F401


def arrays(i, B=2, L=3, C=8, K=4):
    a = lambda *s, dt=torch.float32: OnGpu(s, i, dt)  # noqa: E731
    return dict(x=a(B, L, C), ga=a(B, L, C), gx=a(B, L, C), rate=a(C), h0=a(B, C), reset=a(B, L, dt=torch.bool),
                lengths=a(B, dt=torch.int32), dh=a(B, L, C), saved=a(256, dt=torch.uint8), w=a(C, K), past=a(B, K - 1, C),
                r=a(B, L, C), stats=a(B * L, 2), tok=a(B, C), tok_a=a(B, C), tok_x=a(B, C), state=a(B, C))


def calls(x):
    four, rows = (x["x"], x["ga"], x["gx"], x["rate"]), dict(reset=x["reset"], lengths=x["lengths"])
    return {
        "s5_gated_scan_forward": lambda **kw: api.s5_gated_scan_forward(*four, h0=x["h0"], h_last=True, **rows, **kw),
        "s5_gated_scan_backward": lambda **kw: api.s5_gated_scan_backward(*four, x["dh"], x["saved"], h0=x["h0"], **rows, **kw),
        "s5_gated_scan_step": lambda **kw: api.s5_gated_scan_step(x["tok"], x["tok_a"], x["tok_x"], x["rate"], x["state"], **kw),
        "s5_short_conv_forward": lambda **kw: api.s5_short_conv_forward(x["x"], x["w"], x["rate"], "silu", x["past"], True, **rows, **kw),
        "s5_short_conv_backward": lambda **kw: api.s5_short_conv_backward(x["x"], x["w"], x["dh"], x["rate"], "silu", x["past"], **rows, **kw),
        "s5_short_conv_step": lambda **kw: api.s5_short_conv_step(x["tok"], x["w"], x["past"], x["rate"], "silu", **kw),
        "s5_add_layernorm": lambda **kw: api.s5_add_layernorm(x["x"], x["rate"], x["rate"], x["r"], saved=x["stats"], **kw),
        "s5_add_layernorm_backward": lambda **kw: api.s5_add_layernorm_backward(x["x"], x["dh"], x["stats"], x["rate"], x["rate"], x["r"], **kw),
    }


NAMES = list(calls(arrays(0)))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("index", [0, 1])
def test_the_arrays_device_is_current_at_the_launch(world, name, index):  # noqa: F811
    calls(arrays(index))[name]()
    assert world.calls == [(name, index)] and world.current == 0


@pytest.mark.parametrize("name", NAMES)
def test_the_device_is_given_back_after_an_error(world, name):  # noqa: F811
    x = arrays(1)
    x["rate"] = OnGpu((9, 9), 1)
    with pytest.raises((ValueError, IndexError)):
        calls(x)[name]()
    assert world.current == 0 and world.calls == []


@pytest.mark.parametrize("name,odd", [("s5_gated_scan_forward", "gx"), ("s5_gated_scan_forward", "reset"), ("s5_gated_scan_backward", "saved"),
                                      ("s5_gated_scan_step", "state"), ("s5_short_conv_forward", "past"), ("s5_short_conv_backward", "lengths"),
                                      ("s5_short_conv_step", "w"), ("s5_add_layernorm", "r"), ("s5_add_layernorm_backward", "stats")])
def test_arrays_of_two_devices_are_refused(world, name, odd):  # noqa: F811
    x = arrays(0)
    x[odd] = OnGpu(tuple(x[odd].shape), 1, x[odd].dtype)
    with pytest.raises(ValueError, match="is on cuda:"):
        calls(x)[name]()
    assert world.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_belongs_to_its_stream(world, name):  # noqa: F811
    x = arrays(0)
    side = Stream(0, 22)
    out = returned(calls(x)[name](stream=side))
    assert world.handles == [22] and world.stream is world.home
    assert world.made and all(t.made_on is side for t in world.made)
    for t in out:
        assert not any(t is u for u in world.made) or t.users == [world.home]
    used = [t for t in x.values() if side in t.users]
    assert used and all(t.users == [side] * len(t.users) for t in used)


@pytest.mark.parametrize("name", NAMES)
def test_the_callers_own_stream_needs_no_records(world, name):  # noqa: F811
    x = arrays(0)
    calls(x)[name](stream=Stream(0, 11))
    assert world.handles == [11] and not any(t.users for t in [*x.values(), *world.made])


def test_the_flag_is_reported(monkeypatch):
    class Lib:
        def s5_gated_scan_fault(self):
            return self.code

    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import gated_recurrence
    lib = Lib()
    monkeypatch.setattr(_native, "lib", lambda: lib)
    for lib.code, want in ((0, False), (1, True)):
        assert api.s5_gated_scan_fault() is want
    with pytest.raises(RuntimeError, match="ran out"):
        gated_recurrence.finished()
    lib.code = -1
    with pytest.raises(api.S5Error, match="could not be read"):
        api.s5_gated_scan_fault()
