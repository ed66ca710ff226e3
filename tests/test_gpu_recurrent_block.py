"""GPU tests of the recurrent block's calls as they are used together: the example's streaming and gradients, other
streams, captured graphs that share a workspace."""
import os
import sys

import pytest
import torch

from diagonal_state_space_gb300 import api

from _recurrent_gpu import same

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
CYCLES = 100_000_000          # about 50 ms of waiting


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 2e-2)])
def test_streaming_goes_on_where_the_prompt_ended(dtype, tol):
    """Two layers of a dozen roundings each to 2^-24 and matrix products of sums of 96: 1e-5; to bf16 about five roundings
    of 2^-8 a layer that the two ways share but for their order, rel-L2 2e-2."""
    import gated_recurrence
    assert gated_recurrence.prompt_and_stream(dtype=dtype) < tol


def _reference(m, x, reset, dy):
    """The example's stack in float64 with torch's gradients."""
    layers = [{n: p.double().clone().requires_grad_() for n, p in layer.items()} for layer in m.layers]
    x0 = x.double().clone().requires_grad_()
    total, delta = None, x0
    B, L, _ = x.shape
    age = torch.full((B, L), m.taps, dtype=torch.long, device=x.device)
    for t in range(L):
        prev = age[:, t - 1] + 1 if t else torch.full((B,), m.taps, dtype=torch.long, device=x.device)
        age[:, t] = torch.where(reset[:, t], 0, prev)
    for p in layers:
        total = delta if total is None else total + delta
        c = total - total.mean(-1, keepdim=True)
        n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * p["norm"] + p["shift"]
        u, side = n @ p["w_in"].t(), n @ p["w_side"].t()
        line = torch.nn.functional.pad(u, (0, 0, m.taps - 1, 0))
        v = p["bias"]
        for back in range(m.taps):
            at = m.taps - 1 - back
            v = v + p["conv"][:, at] * line[:, at:at + L] * (age >= back)[..., None]
        v = v * torch.sigmoid(v)
        r, s = torch.sigmoid(v @ p["w_a"].t()), torch.sigmoid(v @ p["w_x"].t())
        la = -torch.nn.functional.softplus(p["lam"]) * r
        a, q = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
        a, q = torch.where(reset[..., None], 0.0, a), torch.where(reset[..., None], 1.0, q)
        h, hs = torch.zeros(B, v.shape[-1], dtype=torch.float64, device=x.device), []
        for t in range(L):
            h = a[:, t] * h + q[:, t] * s[:, t] * v[:, t]
            hs.append(h)
        delta = (torch.stack(hs, 1) * torch.nn.functional.silu(side)) @ p["w_out"].t()
    y = total + delta
    (y * dy.double()).sum().backward()
    return y.detach(), [{n: p.grad for n, p in layer.items()} for layer in layers], x0.grad


def test_gradients_of_the_example_are_those_of_float64():
    import gated_recurrence
    gen = torch.Generator(device="cuda").manual_seed(5)
    m = gated_recurrence.GatedStack(24, 40, seed=4)
    x = torch.randn(2, 75, 24, generator=gen, device="cuda")
    dy = torch.randn(2, 75, 24, generator=gen, device="cuda")
    reset = torch.rand(2, 75, generator=gen, device="cuda") < 0.06
    y, _, kept = m.forward(x, reset=reset, keep=True)
    grads, dx = m.backward(kept, dy)
    gated_recurrence.finished()
    wy, wg, wx = _reference(m, x, reset, dy)
    # rel-L2: forward and backward are some 100 operations deep, each off by a few 2^-24, in sums of up to 150 terms
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y, wy) < 1e-5 and rel(dx, wx) < 5e-5
    for got, want in zip(grads, wg):
        for n in want:
            assert rel(got[n], want[n]) < 5e-5, n


def test_the_example_trains():
    import gated_recurrence
    losses = gated_recurrence.train(steps=2, L=100)
    assert len(losses) == 2 and all(v == v and abs(v) < 1e6 for v in losses)


def make(B=2, L=300, C=128):
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, ga, gx, dh = (r(B, L, C).bfloat16() for _ in range(4))
    past = r(B, 3, C).bfloat16()
    rate, w, b, h0 = torch.rand(C, generator=gen, device="cuda"), r(C, 4), r(C), r(B, C)
    reset = torch.rand(B, L, generator=gen, device="cuda") < 0.02
    saved, stats = api.new_gated_scan_saved(x), api.new_layernorm_saved(x)
    api.s5_gated_scan_forward(x, ga, gx, rate, h0=h0, reset=reset, saved=saved)
    api.s5_add_layernorm(x, b, b, residual=ga, saved=stats)
    tok = [t[:, 0].contiguous() for t in (x, ga, gx)]
    states, pasts = [h0.clone() for _ in range(2)], [past.clone() for _ in range(2)]     # a call each
    there = lambda d: [t for t in d.values() if t is not None]  # noqa: E731
    return {
        "scan": lambda **kw: list(api.s5_gated_scan_forward(x, ga, gx, rate, h0=h0, h_last=True, reset=reset, **kw)),
        "scan_backward": lambda **kw: there(api.s5_gated_scan_backward(x, ga, gx, rate, dh, saved, h0=h0, reset=reset, **kw)),
        "scan_step": lambda **kw: [api.s5_gated_scan_step(*tok, rate, states.pop(), **kw)],
        "conv": lambda **kw: list(api.s5_short_conv_forward(x, w, b, "silu", past=past, past_out=True, reset=reset, **kw)),
        "conv_backward": lambda **kw: there(api.s5_short_conv_backward(x, w, dh, b, "silu", past=past, reset=reset, **kw)),
        "conv_step": lambda **kw: [api.s5_short_conv_step(tok[0], w, pasts.pop(), b, "silu", **kw)],
        "norm": lambda **kw: list(api.s5_add_layernorm(x, b, b, residual=ga, **kw)),
        "norm_backward": lambda **kw: there(api.s5_add_layernorm_backward(x, dh, stats, b, b, residual=ga, dtotal=gx, **kw)),
    }


NAMES = ["scan", "scan_backward", "scan_step", "conv", "conv_backward", "conv_step", "norm", "norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """The same values, in memory that queued work of the current stream still uses left alone."""
    call = make()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    sizes = {t.numel() * t.element_size() for t in want} | {
        api.s5_gated_scan_workspace_size(2, 300, 128), api.s5_short_conv_workspace_size(128, 4), api.s5_add_layernorm_workspace_size(128)}
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side.wait_stream(torch.cuda.current_stream())
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(CYCLES)
    late = [b.clone() for b in blocks]
    del blocks
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert same(list(got), want)
    assert all((b == 7).all() for b in late)


@pytest.mark.parametrize("name", ["scan_backward", "conv_backward", "norm_backward"])
def test_captured_graphs_share_a_workspace(name):
    """Two graphs of the same call with one workspace, replayed in turn, after eager calls with it."""
    call = make()[name]
    work = torch.empty(max(api.s5_gated_scan_workspace_size(2, 300, 128), api.s5_short_conv_workspace_size(128, 4),
                           api.s5_add_layernorm_workspace_size(128)), dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in call(workspace=work)]
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = call(workspace=work)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            for t in out:
                t.zero_()
            work.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert same(list(out), want)


def test_a_captured_step_goes_on_from_its_state():
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = [torch.randn(3, 64, generator=gen, device="cuda") for _ in range(3)]
    rate, w = torch.rand(64, generator=gen, device="cuda"), torch.randn(64, 4, generator=gen, device="cuda")

    def run(state, past):
        c = api.s5_short_conv_step(x[0], w, past, activation="silu")
        return api.s5_gated_scan_step(c, x[1], x[2], rate, state)

    state, past = torch.zeros(3, 64, device="cuda"), torch.zeros(3, 3, 64, device="cuda")
    want = [run(state, past).clone() for _ in range(5)]
    state2, past2 = torch.zeros_like(state), torch.zeros_like(past)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = run(state2, past2)
    state2.zero_(), past2.zero_()
    for w_ in want:
        g.replay()
        torch.cuda.synchronize()
        assert same(h, w_)
    assert same(state, state2) and same(past, past2)


def test_two_streams_at_once():
    """The same calls on two streams side by side, each with a workspace of its own."""
    c = make()
    want = {n: [t.clone() for t in c[n]()] for n in ("scan", "scan_backward", "conv_backward", "norm_backward")}
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        for s in streams:
            for n in want:
                got.append((n, c[n](stream=s)))
    torch.cuda.synchronize()
    assert all(same(list(out), want[n]) for n, out in got)
    assert not api.s5_gated_scan_fault()


FIRST = """
import torch
from diagonal_state_space_gb300 import api
gen = torch.Generator(device="cuda").manual_seed(1)
x, a, g, dh = (torch.randn(2, 600, 72, generator=gen, device="cuda") for _ in range(4))
rate, w, b = torch.rand(72, generator=gen, device="cuda"), torch.randn(72, 5, generator=gen, device="cuda"), torch.randn(72, generator=gen, device="cuda")
def run():
    stats, saved = api.new_layernorm_saved(x), api.new_gated_scan_saved(x)
    n, total = api.s5_add_layernorm(x, b, b, residual=a, saved=stats)
    c = api.s5_short_conv_forward(n, w, bias=b, activation="silu")
    h = api.s5_gated_scan_forward(c, a, g, rate, saved=saved)
    d = api.s5_gated_scan_backward(c, a, g, rate, dh, saved)
    v = api.s5_short_conv_backward(n, w, d["dx"], bias=b, activation="silu")
    m = api.s5_add_layernorm_backward(x, v["dx"], stats, b, b, residual=a, dtotal=dh)
    return [n, total, c, h] + [t for u in (d, v, m) for t in u.values() if t is not None]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(out, run()))
assert not api.s5_gated_scan_fault()
"""


def test_the_first_calls_of_a_process_can_be_captured():
    import subprocess
    res = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
