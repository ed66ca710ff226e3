"""GPU test of calls on another stream than the current one: memory that queued work of the current stream still
uses is not written by the call, and what the call returns is not overwritten while it is read."""
import pytest
import torch

from diagonal_state_space_gb300 import api, init

pytestmark = pytest.mark.gpu
B, L, H, D = 2, 256, 4, 128
CYCLES = 100_000_000          # about 50 ms of waiting


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def make():
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, do = (r(B, L, H, D).bfloat16() for _ in range(4))
    k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
    x = dict(q=q, k=k, v=v, do=do, g=-torch.rand(B, L, H, device="cuda"), beta=torch.rand(B, L, H, device="cuda"))
    x["pos"] = torch.arange(L, device="cuda").expand(B, L).contiguous()
    x["freq"] = torch.from_numpy(init.rotary_frequencies(D)[0]).cuda()
    x["w"] = torch.ones(D, device="cuda")
    x["saved"] = api.new_delta_saved(q, v)
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    api.s5_delta_forward(*five, saved=x["saved"])
    tok = [t[:, 0].contiguous() for t in five]
    states = [torch.zeros(B, H, D, D, device="cuda") for _ in range(2)]      # a call each
    return {
        "forward": lambda **kw: list(api.s5_delta_forward(*five, s_last=True, **kw)),
        "backward": lambda **kw: [t for t in api.s5_delta_backward(*five, x["do"], x["saved"], **kw).values() if t is not None],
        "step": lambda **kw: [api.s5_delta_step(*tok, states.pop(), **kw)],
        "rotary": lambda **kw: [api.s5_rotary(x["q"], x["pos"], x["freq"], **kw)],
        "norm": lambda **kw: list(api.s5_qk_norm_rotary(x["q"], x["k"], x["pos"], x["freq"], **kw)),
        "norm_backward": lambda **kw: list(api.s5_qk_norm_rotary_backward(
            x["q"], x["k"], x["do"], x["do"], x["pos"], x["freq"], q_weight=x["w"], k_weight=x["w"], **kw).values()),
    }


def fill_and_free(sizes):
    """Blocks of these sizes, filled; a queued copy of each that runs late; then they are free for the allocator."""
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(CYCLES)
    return [b.clone() for b in blocks]


@pytest.mark.parametrize("name", ["forward", "backward", "step", "rotary", "norm", "norm_backward"])
def test_memory_still_in_use_on_the_current_stream_is_left_alone(name):
    call = make()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    work = [api.s5_delta_workspace_size(B, L, H, D, D), api.s5_delta_workspace_size(B, L, H, D, D, True)]
    sizes = {t.numel() * t.element_size() for t in want} | set(work)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side.wait_stream(torch.cuda.current_stream())
    copies = fill_and_free(sorted(sizes))
    got = call(stream=side)                  # runs at once; the copies above have yet to read the freed blocks
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_freed_while_the_current_stream_reads_them():
    call = make()["rotary"]
    want = call()[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(CYCLES)
    late = y.clone()
    del y
    with torch.cuda.stream(side):            # the side stream may not get that memory yet
        for _ in range(4):
            torch.full_like(want, 5.0)
    torch.cuda.synchronize()
    assert torch.equal(late, want)


def test_arrays_freed_while_the_call_reads_them():
    """Temporaries of the current stream given to a call on a busy side stream."""
    x = torch.randn(B, L, H, D, device="cuda").bfloat16()
    pos = torch.arange(L, device="cuda").expand(B, L).contiguous()
    freq = torch.from_numpy(init.rotary_frequencies(D)[0]).cuda()
    want = api.s5_rotary(x, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    temporary = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = api.s5_rotary(temporary, pos, freq, stream=side)
    del temporary
    for _ in range(4):
        torch.full_like(x, 5.0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
