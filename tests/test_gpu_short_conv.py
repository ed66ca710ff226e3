"""GPU tests of the short causal convolution against float64, value by value (tests/_recurrent_ref.py derives the bounds)."""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import api

import _recurrent_ref as ref
from _recurrent_gpu import TYPES, close, host, rnd, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def make(B, L, C, K, kind, bias=True, past=False, marks=0.0, ragged=False, seed=0):
    rng = np.random.default_rng(seed)
    return dict(x=rnd((B, L, C), kind, seed + 1)[0], w=rnd((C, K), "f32", seed + 2)[0], bias=rnd((C,), "f32", seed + 3)[0] if bias else None,
                past=rnd((B, K - 1, C), kind, seed + 4)[0] if past else None, dy=rnd((B, L, C), kind, seed + 5)[0],
                dlast=rnd((B, K - 1, C), kind, seed + 6)[0] if past else None,
                reset=torch.from_numpy(rng.random((B, L)) < marks).cuda() if marks else None,
                lengths=torch.from_numpy(rng.integers(0, L + 1, B)).to(torch.int32).cuda() if ragged else None)


def run(t, act):
    kw = dict(bias=t["bias"], activation=act, past=t["past"], reset=t["reset"], lengths=t["lengths"])
    y, last = api.s5_short_conv_forward(t["x"], t["w"], past_out=True, **kw)
    g = api.s5_short_conv_backward(t["x"], t["w"], t["dy"], dpast_out=t["dlast"], **kw)
    return dict(g, y=y, past_out=last)


def want(t, act):
    v = {n: host(a) for n, a in t.items() if n not in ("reset", "lengths")}
    reset = None if t["reset"] is None else t["reset"].bool().cpu().numpy()
    lengths = None if t["lengths"] is None else t["lengths"].cpu().numpy()
    return ref.conv(v["x"], v["w"], v["bias"], act == "silu", v["past"], reset, lengths, v["dy"], v["dlast"])


def check(t, act):
    got, exp = run(t, act), want(t, act)
    for n, e in exp.items():
        close(got[n], e, n)
    assert (got["dbias"] is None) == (t["bias"] is None) and (got["dpast"] is None) == (t["past"] is None)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("K", range(2, 9))
@pytest.mark.parametrize("C", [1, 6, 132])
def test_taps_and_channels(C, K, act, kind):
    check(make(2, 37, C, K, kind, bias=K % 2 == 0, past=act is None, seed=C + K), act)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("B,L,C", [(1, 1, 4), (3, 2, 8), (2, 7, 5), (1, 8, 128), (2, 65, 130), (1, 700, 12), (300, 9, 8), (2, 600, 1030), (40, 200, 260)])
def test_lengths_of_sequences(B, L, C, kind):
    check(make(B, L, C, 4, kind, past=True, seed=L), "silu")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("L", [3, 50, 200])
@pytest.mark.parametrize("marks,ragged", [(0.05, False), (0.5, False), (1.0, False), (0.0, True), (0.2, True)])
def test_resets_and_lengths(L, K, marks, ragged, kind):
    check(make(5, L, 20, K, kind, past=True, marks=marks, ragged=ragged, seed=L + K), "silu")


def test_lengths_outside_the_row_are_taken_into_it():
    t = make(4, 20, 8, 4, "f32", past=True, seed=1)
    t["lengths"] = torch.tensor([-3, 0, 20, 1000], dtype=torch.int32, device="cuda")
    check(t, None)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [None, "silu"])
def test_nothing_behind_a_reset_or_an_end_is_seen(act, kind):
    t = make(2, 100, 20, 4, kind, past=True, seed=9)
    t["reset"] = torch.zeros(2, 100, dtype=torch.uint8, device="cuda")
    t["reset"][:, 30] = 1
    t["reset"][0, 61] = 255
    t["reset"][1, 0] = 1
    t["lengths"] = torch.tensor([90, 100], dtype=torch.int32, device="cuda")
    clean = run(t, act)
    dirty = {n: a if a is None else a.clone() for n, a in t.items()}
    for n in ("x", "dy"):
        dirty[n][0, 30:61] = float("nan")
        dirty[n][0, 90:] = float("inf")
    dirty["past"][1] = float("nan")
    got = run(dirty, act)
    rest = torch.ones(2, 100, dtype=torch.bool)
    rest[0, 30:61] = False
    for n in ("y", "dx"):
        assert torch.equal(got[n][rest.cuda()], clean[n][rest.cuda()]), n
        assert torch.isnan(got[n][0, 30:61]).all(), n
        assert torch.count_nonzero(got[n][0, 90:]) == 0
    assert same(got["past_out"], clean["past_out"]) and same(got["dpast"], clean["dpast"])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("K", range(2, 9))
@pytest.mark.parametrize("B,C", [(1, 1), (96, 1024), (3, 330), (5, 7)])
def test_step(B, C, K, kind):
    t = make(B, 1, C, K, kind, past=True, seed=B + C)
    exp = want(t, "silu")
    state, x = t["past"].clone(), t["x"][:, 0].contiguous()
    y = api.s5_short_conv_step(x, t["w"], state, bias=t["bias"], activation="silu")
    close(y, (exp["y"][0][:, 0], exp["y"][1][:, 0]), "y")
    assert np.array_equal(host(state), exp["past_out"][0])
    again = t["past"].clone()
    assert api.s5_short_conv_step(x, t["w"], again, bias=t["bias"], activation="silu", y=x) is x
    assert torch.equal(x, y) and torch.equal(again, state)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("cut", [1, 2, 40, 99])
def test_parts_of_a_sequence_are_the_whole(cut, kind):
    t = make(2, 100, 24, 4, kind, past=True, marks=0.1, seed=cut)
    exp = want(t, "silu")
    kw = dict(bias=t["bias"], activation="silu")
    part = lambda n, s: t[n][:, s].contiguous()  # noqa: E731
    a, b = slice(0, cut), slice(cut, 100)
    ya, mid = api.s5_short_conv_forward(part("x", a), t["w"], past=t["past"], past_out=True, reset=part("reset", a), **kw)
    state = mid.clone()
    yb, last = api.s5_short_conv_forward(part("x", b), t["w"], past=state, past_out=state, reset=part("reset", b), **kw)
    assert last is state                 # in place
    close(torch.cat([ya, yb], 1), exp["y"], "y")
    assert np.array_equal(host(last), exp["past_out"][0])
    if kind == "f32":                    # what passes between the calls is rounded to the type
        gb = api.s5_short_conv_backward(part("x", b), t["w"], part("dy", b), past=mid, dpast_out=t["dlast"], reset=part("reset", b), **kw)
        ga = api.s5_short_conv_backward(part("x", a), t["w"], part("dy", a), past=t["past"], dpast_out=gb["dpast"], reset=part("reset", a), **kw)
        close(torch.cat([ga["dx"], gb["dx"]], 1), exp["dx"], "dx")
        close(ga["dpast"], exp["dpast"], "dpast")
        close(ga["dweight"] + gb["dweight"], exp["dweight"], "dweight")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C,gap", [(64, 32), (40, 2), (40, 1)])
def test_views_of_a_fused_projection(C, gap, kind):
    t = make(2, 90, C, 4, kind, seed=8)
    fused = torch.full((2, 90, 2 * C + gap), float("nan"), device="cuda", dtype=TYPES[kind])
    v = dict(t)
    for i, n in enumerate(("x", "dy")):
        v[n] = fused[..., i * C:(i + 1) * C]
        v[n].copy_(t[n])
    exp, got = want(t, "silu"), run(v, "silu")
    for n, e in exp.items():
        close(got[n], e, n)
    wide = torch.full((2, 90, C + 16), 7.0, device="cuda", dtype=TYPES[kind])
    close(api.s5_short_conv_forward(v["x"], t["w"], bias=t["bias"], activation="silu", y=wide[..., :C]), exp["y"], "y")
    assert (wide[..., C:] == 7.0).all()


def test_empty_calls():
    for B, L in ((0, 5), (2, 0)):
        t = make(B, L, 8, 4, "bf16", past=True, seed=1)
        got = run(t, "silu")
        assert got["y"].shape == (B, L, 8) and torch.equal(got["past_out"], t["past"]) and torch.equal(got["dpast"], t["dlast"])
        assert torch.count_nonzero(got["dweight"]) == 0 and torch.count_nonzero(got["dbias"]) == 0


def test_equal_inputs_give_equal_bits():
    t = make(2, 3000, 128, 4, "bf16", marks=0.01, seed=11)
    first = run(t, "silu")
    for _ in range(5):
        assert same(run(t, "silu"), first)


def test_offsets_past_32_bits():
    L, C, ld = 70_000, 8, 32_000
    big = torch.empty(L * ld, device="cuda", dtype=torch.bfloat16)
    x = big.as_strided((1, L, C), (L * ld, ld, 1))
    t = make(1, L, C, 4, "bf16", seed=12)
    x.copy_(t["x"])
    a, b = run(dict(t, x=x), "silu"), run(t, "silu")
    assert same(a, b)
