"""Host checks of which device and stream the mixer's calls launch on, with stand-ins for tensors of several
GPUs, for streams and for the library: the device that is current when the library is entered has to be the
tensors', and what a call makes has to belong to its stream."""
import contextlib

import pytest
import torch

from diagonal_state_space_gb300 import _native, api


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""

    @staticmethod
    def __new__(cls, shape, index, dtype=torch.float32):
        t = torch.Tensor._make_subclass(cls, torch.zeros(shape, dtype=dtype))
        t.index, t.made_on, t.users = index, None, []
        return t

    def record_stream(self, stream):
        self.users.append(stream)

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        with torch._C.DisableTorchFunctionSubclass():
            return func(*args, **(kwargs or {}))


class Stream:
    def __init__(self, index, handle):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


@pytest.fixture
def world(monkeypatch):
    """current: the device; stream: the stream; calls: (entry point, device current at the call); made: what calls
    made; handles: the streams that they launched on."""
    class World:
        pass

    w = World()
    w.current, w.calls, w.made, w.handles = 0, [], [], []
    w.home = w.stream = Stream(0, 11)

    @contextlib.contextmanager
    def device(d):
        before, w.current = w.current, torch.device(d).index
        try:
            yield
        finally:
            w.current = before

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 256
            return lambda *a: w.calls.append((name, w.current)) or w.handles.append(a[-1]) or 0

    @contextlib.contextmanager
    def stream(s):
        before, w.stream = w.stream, s
        try:
            yield
        finally:
            w.stream = before

    def new(shape, index, dtype):
        t = OnGpu(tuple(shape), index, dtype)
        t.made_on = w.stream
        w.made.append(t)
        return t

    real_empty = torch.empty
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: w.stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: w.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_native, "lib", lambda: Lib())
    monkeypatch.setattr(api, "_raw_stream", lambda index: 0)

    def empty(*shape, dtype=torch.float32, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        if device is None or torch.device(device).type != "cuda":
            return real_empty(shape, dtype=dtype)
        return new(shape, torch.device(device).index, dtype)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(api, "_new", lambda t: new(t.shape, t.index, t.dtype))
    if _native._marshal is None:
        class Native:                        # leaves every call to Python
            def __getattr__(self, name):
                return lambda *a: None
        monkeypatch.setattr(_native, "marshal", lambda: Native())
    return w


def arrays(i, B=2, L=3, Hk=1, Hv=2, D=8):
    a = lambda *s, dt=torch.float32: OnGpu(s, i, dt)  # noqa: E731
    return dict(q=a(B, L, Hk, D), k=a(B, L, Hk, D), v=a(B, L, Hv, D), g=a(B, L, Hv), beta=a(B, L, Hv), do=a(B, L, Hv, D),
                saved=a(256, dt=torch.uint8), pos=a(B, L, dt=torch.int64), freq=a(4, dt=torch.float64), w=a(D),
                state=a(B, Hv, D, D))


def calls(x):
    tok = {n: OnGpu(x[n].shape[:1] + x[n].shape[2:], x[n].index) for n in ("q", "k", "v", "g", "beta")}
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    return {
        "s5_delta_forward": lambda **kw: api.s5_delta_forward(*five, s_last=True, **kw),
        "s5_delta_backward": lambda **kw: api.s5_delta_backward(*five, x["do"], x["saved"], **kw),
        "s5_delta_step": lambda **kw: api.s5_delta_step(*tok.values(), x["state"], **kw),
        "s5_rotary": lambda **kw: api.s5_rotary(x["q"], x["pos"], x["freq"], **kw),
        "s5_qk_norm_rotary": lambda **kw: api.s5_qk_norm_rotary(x["q"], x["k"], x["pos"], x["freq"], q_weight=x["w"], **kw),
        "s5_qk_norm_rotary_backward": lambda **kw: api.s5_qk_norm_rotary_backward(
            x["q"], x["k"], x["q"], x["k"], x["pos"], x["freq"], q_weight=x["w"], **kw),
    }


NAMES = list(calls(arrays(0)))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("index", [0, 1])
def test_the_arrays_device_is_current_at_the_launch(world, name, index):
    calls(arrays(index))[name]()
    assert world.calls == [(name, index)] and world.current == 0


@pytest.mark.parametrize("name", NAMES)
def test_the_device_is_given_back_after_an_error(world, name):
    x = arrays(1)
    x["freq"] = OnGpu((4,), 1)               # not float64
    x["g"] = OnGpu((9, 9), 1)
    with pytest.raises((ValueError, IndexError)):
        calls(x)[name]()
    assert world.current == 0 and world.calls == []


@pytest.mark.parametrize("name,odd", [("s5_delta_forward", "k"), ("s5_delta_forward", "beta"), ("s5_delta_backward", "do"),
                                      ("s5_delta_backward", "saved"), ("s5_delta_step", "state"), ("s5_rotary", "pos"),
                                      ("s5_rotary", "freq"), ("s5_qk_norm_rotary", "w"), ("s5_qk_norm_rotary", "k"),
                                      ("s5_qk_norm_rotary_backward", "freq")])
def test_arrays_of_two_devices_are_refused(world, name, odd):
    x = arrays(0)
    x[odd] = OnGpu(tuple(x[odd].shape), 1, x[odd].dtype)
    with pytest.raises(ValueError, match="is on cuda:"):
        calls(x)[name]()
    assert world.calls == []


def returned(out):
    out = list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]
    return [t for t in out if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_belongs_to_its_stream(world, name):
    x = arrays(0)
    side = Stream(0, 22)
    out = returned(calls(x)[name](stream=side))
    assert world.handles == [22] and world.stream is world.home
    assert world.made and all(t.made_on is side for t in world.made)
    for t in world.made:                    # the caller's stream is known for what it gets, and only for that
        assert t.users == ([world.home] if any(t is u for u in out) else [])
    used = [t for t in x.values() if side in t.users]
    assert used and all(t.users == [side] * len(t.users) for t in used)


@pytest.mark.parametrize("name", NAMES)
def test_the_callers_own_stream_needs_no_records(world, name):
    x = arrays(0)
    calls(x)[name](stream=Stream(0, 11))
    assert world.handles == [11] and not any(t.users for t in [*x.values(), *world.made])


def test_a_stream_of_another_device_is_refused(world):
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        calls(arrays(0))["s5_rotary"](stream=Stream(1, 22))
    assert world.calls == [] and world.current == 0
