"""GPU tests of the rotation and of the norms with it, against float64.

Tolerances (rel-L2).  An fp32 result passes at most 16 roundings of 2^-24 (sum
of squares over a group of lanes, root, weight, angle of 2^-25 half turns =
2^-23.3 radians, products); a weight's gradient sums the rows in parts, up to
100 in a row in each: 64.  bf16 outputs get one rounding of 2^-8 besides.
"""
import numpy as np
import pytest
import torch

from diagonal_state_space_gb300 import _native, api, init

import _mixer_ref as ref
from _parity import check

pytestmark = pytest.mark.gpu

F32, DW, BF16 = 16 * 2.0 ** -24, 64 * 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def host(t):
    return t.double().cpu().numpy()


def rnd(shape, dt, seed):
    t = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).cuda().to(dt)
    return t, host(t)


def tol(dt):
    return F32 + (BF16 if dt == torch.bfloat16 else 0)


# D, rot: vectors of every width, parts of the head, whole warps, several slots per lane
HEADS = [(128, 128), (128, 64), (64, 64), (256, 256), (256, 64), (80, 48), (80, 40), (96, 48), (2, 2), (6, 4), (18, 6),
         (254, 250), (36, 0), (16, 16), (32, 8)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", HEADS)
def test_rotary(D, rot, layout, dt):
    x, vx = rnd((2, 13, 3, D), dt, D + rot)
    pos = torch.randint(0, 1 << 20, (2, 13), generator=torch.Generator().manual_seed(1)).cuda()
    if rot:
        freq, _ = init.rotary_frequencies(rot)
        fr = torch.from_numpy(freq).cuda()
    else:
        freq, fr, pos = np.zeros(0), None, None
    p = np.zeros((2, 13)) if pos is None else pos.cpu().numpy()
    y = api.s5_rotary(x, pos, fr, layout=layout, amplitude=1.3)
    check(host(y), ref.turn(vx, p, freq, layout, 1.3), tol(dt), "y")
    if rot < D:
        assert torch.equal(y[..., rot:], x[..., rot:])
    back = api.s5_rotary(x, pos, fr, layout=layout, amplitude=1.3, inverse=True)
    check(host(back), ref.turn(vx, p, freq, layout, 1.3, back=True), tol(dt), "transposed")


@pytest.mark.parametrize("start", [0, 1_000_000, (1 << 31) - 20, (1 << 40) + 5, -77])
def test_rotary_positions(start):
    """Far positions: float64 products are off by position * frequency * 2^-53 themselves, 2^-13 radians at 2^40; the
    expectation there comes from exact integer products."""
    x, vx = rnd((9, 2, 64), torch.float32, 5)
    pos = torch.arange(9, device="cuda") + start
    freq, _ = init.rotary_frequencies(64, base=500000.0, scaling="by_parts", factor=8.0, trained=8192)
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    turns = np.array([[float((Fraction(int(p)) * Fraction(float(f)) / two_pi) % 1) for f in freq] for p in pos.tolist()])
    w = np.exp(2j * np.pi * turns)[:, None, :]
    c = (vx[..., :32] + 1j * vx[..., 32:]) * w
    y = api.s5_rotary(x, pos, torch.from_numpy(freq).cuda())
    check(host(y), np.concatenate([c.real, c.imag], -1), F32, "y")


def test_rotary_negative_and_large_frequencies():
    x, vx = rnd((7, 1, 8), torch.float32, 6)
    freq = np.array([-0.25, 100.0, 7e-9, 0.0])
    pos = torch.arange(7, device="cuda") * 3
    y = api.s5_rotary(x, pos, torch.from_numpy(freq).cuda())
    check(host(y), ref.turn(vx, pos.cpu().numpy(), freq, "half", 1.0), F32, "y")


QK = [(1, 1, 16, 16, 128, 128, "rms"), (3, 7, 8, 2, 128, 64, "l2"), (2, 50, 4, 1, 64, 64, None), (2, 9, 3, 5, 80, 48, "rms"),
      (1, 33, 9, 0, 128, 128, "l2"), (1, 33, 0, 3, 96, 48, "rms"), (2, 11, 1, 1, 18, 6, "rms"), (1, 5, 2, 2, 256, 256, "l2"),
      (1, 700, 12, 4, 128, 128, "rms")]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("case", QK)
def test_qk_norm_rotary_and_backward(case, layout, weighted, dt):
    B, L, Hq, Hk, D, rot, kind = case
    freq, amp = init.rotary_frequencies(rot, scaling="by_parts", factor=4.0, trained=2048)
    fr, pos = torch.from_numpy(freq).cuda(), torch.arange(L, device="cuda").repeat(B, 1) + 1000
    p = pos.cpu().numpy()
    x = {n: rnd((B, L, h, D), dt, i) for i, (n, h) in enumerate((("q", Hq), ("k", Hk), ("gq", Hq), ("gk", Hk)))}
    w = {n: rnd((D,), torch.float32, i + 9) if weighted else (None, None) for i, n in enumerate("qk")}
    kw = dict(norm=kind, eps=1e-5, q_weight=w["q"][0], k_weight=w["k"][0], layout=layout, amplitude=amp)
    q, k = api.s5_qk_norm_rotary(x["q"][0], x["k"][0], pos, fr, **kw)
    g = api.s5_qk_norm_rotary_backward(x["q"][0], x["k"][0], x["gq"][0], x["gk"][0], pos, fr, **kw)
    for n, y, h in (("q", q, Hq), ("k", k, Hk)):
        if h == 0:
            if weighted:
                assert torch.count_nonzero(g["dw" + n]) == 0
            continue
        vx, vw = x[n][1], w[n][1]
        check(host(y), ref.turn(ref.norm(vx, vw, kind, 1e-5)[0], p, freq, layout, amp), tol(dt), n)
        dx, dw = ref.norm_turn_backward(vx, vw, kind, 1e-5, p, freq, layout, amp, x["g" + n][1])
        check(host(g["d" + n]), dx, 2 * F32 + (BF16 if dt == torch.bfloat16 else 0), "d" + n)
        if weighted:
            check(host(g["dw" + n]), dw, DW, "dw" + n)
        else:
            assert g["dw" + n] is None


# Sizes from which on the rows stream through shared memory: several segments a
# token, a last one that is not full, items that do not divide among the warps
BIG = [(2, 4501, 12, 3, 128, 128, "rms", "half"), (1, 8100, 33, 1, 64, 32, "l2", "interleaved"),
       (3, 500, 40, 8, 256, 256, "rms", "interleaved"), (1, 14099, 9, 7, 80, 48, "l2", "half"),
       (1, 37000, 0, 5, 96, 96, "rms", "half"), (1, 19001, 7, 0, 128, 64, None, "interleaved")]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", BIG)
def test_large_qk_norm_rotary_and_backward(case, dt):
    test_qk_norm_rotary_and_backward(case[:-1], case[-1], True, dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_large_rotary_from_and_into_views(dt):
    """Pitches of a fused projection, a larger output, and in place."""
    B, L, H, D = 1, 16007, 9, 128
    fused = torch.full((B, L, 2 * H * D + 64), float("nan"), device="cuda", dtype=dt)
    x = fused[:, :, 64:64 + H * D].unflatten(-1, (H, D))
    x.copy_(torch.randn(B, L, H, D, device="cuda"))
    vx, pos = host(x), torch.arange(L, device="cuda")[None] * 7
    freq = init.rotary_frequencies(128)[0]
    want = ref.turn(vx, pos.cpu().numpy(), freq, "half", 1.0)
    y = api.s5_rotary(x, pos, torch.from_numpy(freq).cuda())
    check(host(y), want, tol(dt), "y")
    wide = torch.zeros(B, L, H * D + 8, device="cuda", dtype=dt)
    api.s5_rotary(x, pos, torch.from_numpy(freq).cuda(), out=wide[:, :, :H * D].unflatten(-1, (H, D)))
    assert torch.equal(wide[:, :, :H * D], y.flatten(-2)) and torch.count_nonzero(wide[:, :, H * D:]) == 0
    api.s5_rotary(x, pos, torch.from_numpy(freq).cuda(), out=x)
    assert torch.equal(x, y) and torch.isnan(fused[:, :, :64]).all() and torch.isnan(fused[:, :, 64 + H * D:]).all()


def test_zero_rows_and_infinities_stay_in_their_rows():
    freq = torch.from_numpy(init.rotary_frequencies(128)[0]).cuda()
    x, _ = rnd((1, 4, 3, 128), torch.bfloat16, 3)
    pos = torch.arange(4, device="cuda")[None]
    want = api.s5_qk_norm_rotary(x, x, pos, freq)[0]
    x[0, 1, 1] = 0
    x[0, 2, 0, 7] = float("inf")
    x[0, 2, 2, 9] = float("nan")
    got = api.s5_qk_norm_rotary(x, x, pos, freq)[0]
    assert torch.count_nonzero(got[0, 1, 1]) == 0
    assert torch.isnan(got[0, 2, 0]).any() and torch.isnan(got[0, 2, 2]).all()
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = keep[2, 2] = False
    assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()])
    g = api.s5_qk_norm_rotary_backward(x[:, :2].contiguous(), x[:, :2].contiguous(), x[:, :2].contiguous(),
                                       x[:, :2].contiguous(), pos[:, :2].contiguous(), freq)
    assert torch.isfinite(g["dq"]).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_views_in_place_stream_and_graph(dt):
    freq = torch.from_numpy(init.rotary_frequencies(64)[0]).cuda()
    B, L, H, D = 2, 19, 4, 128
    pos = torch.arange(L, device="cuda").repeat(B, 1)
    for extra in (0, 3):
        fused = torch.randn(B, L, 2 * H * D + 16 // dt.itemsize + extra, device="cuda").to(dt)
        q = fused[:, :, :H * D].unflatten(-1, (H, D))
        k = fused[:, :, H * D:2 * H * D].unflatten(-1, (H, D))
        want = api.s5_qk_norm_rotary(q.contiguous(), k.contiguous(), pos, freq, norm="l2")
        got = api.s5_qk_norm_rotary(q, k, pos, freq, norm="l2")
        for a, b in zip(want, got):     # an odd pitch adds a row's squares in another order
            check(host(b), host(a), 2 * tol(dt) if extra else 0, "view")
        rest = fused[:, :, 2 * H * D:].clone()
        api.s5_qk_norm_rotary(q, k, pos, freq, norm="l2", q_out=q, k_out=k)
        assert torch.equal(q, got[0]) and torch.equal(k, got[1]) and torch.equal(rest, fused[:, :, 2 * H * D:])
    x = torch.randn(B, L, H, D, device="cuda").to(dt)
    want = api.s5_rotary(x, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.s5_rotary(x, pos, freq, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.s5_rotary(x, pos, freq)
        api.s5_rotary(y, pos, freq, inverse=True, out=y)
    graph.replay()
    torch.cuda.synchronize()
    assert (y.float() - x.float()).norm() <= (2 * BF16 if dt == torch.bfloat16 else 2 * F32) * x.float().norm()
    empty = api.s5_rotary(x[:, :0], pos[:, :0], freq)
    assert empty.shape == (B, 0, H, D)


def test_refuses_wrong_arguments():
    x = torch.zeros(2, 3, 4, 64, device="cuda")
    pos, fr = torch.zeros(2, 3, dtype=torch.int64, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError, match="positions"):
        api.s5_rotary(x, pos[:1], fr)
    with pytest.raises(ValueError, match="int64"):
        api.s5_rotary(x, pos.int(), fr)
    with pytest.raises(ValueError, match="freq"):
        api.s5_rotary(x, pos, fr.float())
    with pytest.raises(api.S5Error):
        api.s5_rotary(x, pos, torch.ones(33, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="k must have shape"):
        api.s5_qk_norm_rotary(x, x[:1], pos, fr)
    with pytest.raises(KeyError):
        api.s5_rotary(x, pos, fr, layout="other")


def test_no_copy_ran_out():
    x = torch.randn(4, 4096, 16, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(4096, device="cuda").expand(4, 4096).contiguous()
    api.s5_rotary(x, pos, torch.ones(64, dtype=torch.float64, device="cuda"))
    assert _native.lib().s5_rotary_fault() == 0
