"""GPU tests that arrays which the calls make are made as torch.empty makes them: filled where torch is told to fill
what is not written yet, and seen by dispatch modes and profilers."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from diagonal_state_space_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def test_buffers_are_filled_where_torch_fills(deterministic):
    x = torch.zeros(2, 70, 8, device="cuda")
    for _ in range(3):                   # whatever the memory held
        junk = torch.zeros(4096, dtype=torch.uint8, device="cuda")
        del junk
        assert torch.isnan(api.new_layernorm_saved(x)).all()
        assert (api.new_gated_scan_saved(x) == 255).all()
    torch.utils.deterministic.fill_uninitialized_memory = False
    try:
        assert api.new_layernorm_saved(x).shape == (140, 2)      # not filled: nothing is said of what it holds
    finally:
        torch.utils.deterministic.fill_uninitialized_memory = True


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.ops = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.ops.append(func)
        return func(*args, **(kwargs or {}))


def calls():
    x = torch.randn(2, 9, 8, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda")
    freq = torch.rand(32, dtype=torch.float64, device="cuda")
    pos = torch.arange(2, device="cuda")
    return {
        "s5_add_layernorm": lambda: api.s5_add_layernorm(x),
        "s5_gated_scan_forward": lambda: api.s5_gated_scan_forward(x, x, None, torch.ones_like(x[0, 0])),
        "s5_rotary": lambda: api.s5_rotary(q, pos, freq),
    }


@pytest.mark.parametrize("name", ["s5_add_layernorm", "s5_gated_scan_forward", "s5_rotary"])
def test_a_dispatch_mode_sees_the_arrays(name):
    call = calls()[name]
    want = call()
    with Seen() as seen:
        got = call()
    assert any(op.overloadpacket in (torch.ops.aten.empty, torch.ops.aten.empty_like) for op in seen.ops)
    assert torch.equal(got, want) and got.is_contiguous() and not got.requires_grad


@pytest.mark.parametrize("name", ["s5_add_layernorm", "s5_gated_scan_forward", "s5_rotary"])
def test_a_profiler_lists_the_arrays(name):
    call = calls()[name]
    call()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        call()
    assert any(e.name in ("aten::empty", "aten::empty_like") for e in prof.events())


def test_arrays_of_inference_mode_are_its_own():
    for name, call in calls().items():
        with torch.inference_mode():
            assert call().is_inference(), name
        assert not call().is_inference(), name
