"""GPU tests of the gated linear recurrence against float64, value by value (tests/_recurrent_ref.py derives the bounds)."""
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


def make(B, L, C, kind, gated=True, h0=False, marks=0.0, ragged=False, seed=0, rates=(1e-3, 4.0)):
    rng = np.random.default_rng(seed)
    t = dict(x=rnd((B, L, C), kind, seed + 1)[0], ga=rnd((B, L, C), kind, seed + 2, 2.0)[0],
             gx=rnd((B, L, C), kind, seed + 3)[0] if gated else None,
             rate=torch.from_numpy(np.exp(rng.uniform(np.log(rates[0]), np.log(rates[1]), C))).float().cuda(),
             h0=rnd((B, C), "f32", seed + 4)[0] if h0 else None, dh=rnd((B, L, C), kind, seed + 5)[0],
             dh_last=rnd((B, C), "f32", seed + 6)[0] if h0 else None,
             reset=torch.from_numpy(rng.random((B, L)) < marks).cuda() if marks else None,
             lengths=torch.from_numpy(rng.integers(0, L + 1, B)).to(torch.int32).cuda() if ragged else None)
    return t


def run(t, normalize=True):
    kw = dict(reset=t["reset"], lengths=t["lengths"], normalize=normalize)
    saved = api.new_gated_scan_saved(t["x"])
    h, last = api.s5_gated_scan_forward(t["x"], t["ga"], t["gx"], t["rate"], h0=t["h0"], h_last=True, saved=saved, **kw)
    g = api.s5_gated_scan_backward(t["x"], t["ga"], t["gx"], t["rate"], t["dh"], saved, h0=t["h0"], dh_last=t["dh_last"], **kw)
    return dict(g, h=h, h_last=last)


def want(t, normalize=True):
    v = {n: host(a) for n, a in t.items() if n not in ("reset", "lengths")}
    reset = None if t["reset"] is None else t["reset"].bool().cpu().numpy()
    lengths = None if t["lengths"] is None else t["lengths"].cpu().numpy()
    return ref.scan(v["x"], v["ga"], v["gx"], v["rate"], v["h0"], reset, lengths, normalize, v["dh"], v["dh_last"])


def check(t, normalize=True):
    got, exp = run(t, normalize), want(t, normalize)
    for n, e in exp.items():
        close(got[n], e, n)
    assert (got["dgate_x"] is None) == (t["gx"] is None) and (got["dh0"] is None) == (t["h0"] is None)
    return got


# one token, tiles of every fill, clusters of 1 to 8, several rounds, channels for 16-byte copies, pairs and single ones
SIZES = [(1, 1, 1), (2, 5, 7), (1, 64, 64), (2, 65, 72), (1, 128, 8), (2, 129, 66), (3, 300, 40), (1, 517, 130), (1, 1030, 16), (2, 2500, 9),
         (1, 2049, 96)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_sequences(size, gated, kind):
    check(make(*size, kind, gated=gated, h0=gated, seed=sum(size)))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", [(2, 5, 8), (3, 200, 40), (2, 1100, 18), (4, 333, 7)])
@pytest.mark.parametrize("marks,ragged", [(0.02, False), (0.5, False), (1.0, False), (0.0, True), (0.1, True)])
def test_resets_and_lengths(size, marks, ragged, kind):
    check(make(*size, kind, h0=True, marks=marks, ragged=ragged, seed=7))


@pytest.mark.parametrize("kind", TYPES)
def test_without_the_root(kind):
    check(make(2, 300, 40, kind, h0=True, marks=0.02, seed=3, rates=(0.1, 4.0)), normalize=False)


@pytest.mark.parametrize("kind,C", [("bf16", 257), ("f32", 258), ("bf16", 264)])
def test_many_sequences(kind, C):
    """More blocks than run at once, each through several tiles."""
    check(make(60, 200, C, kind, h0=True, seed=5))


def test_lengths_outside_the_row_are_taken_into_it():
    t = make(4, 20, 8, "f32", h0=True, seed=1)
    t["lengths"] = torch.tensor([-3, 0, 20, 1000], dtype=torch.int32, device="cuda")
    check(t)


@pytest.mark.parametrize("kind", TYPES)
def test_nothing_behind_a_reset_or_an_end_is_seen(kind):
    """NaN and infinities in a sequence stay in it, and what lies behind a row's end is not read."""
    t = make(2, 300, 40, kind, h0=True, seed=9)
    t["reset"] = torch.zeros(2, 300, dtype=torch.uint8, device="cuda")
    t["reset"][:, 100] = 1
    t["reset"][0, 173] = 255
    t["lengths"] = torch.tensor([250, 300], dtype=torch.int32, device="cuda")
    clean, exp = run(t), want(t)
    dirty = {n: a if a is None else a.clone() for n, a in t.items()}
    for n in ("x", "ga", "gx", "dh"):
        dirty[n][0, 100:173] = float("nan")
        dirty[n][0, 250:] = float("inf")
    dirty["h0"][1] = float("nan")
    got = run(dirty)
    for n in ("h", "dx", "dgate_a", "dgate_x"):
        rest = torch.ones(2, 300, dtype=torch.bool)
        rest[0, :173] = False        # the gradients of 0 .. 99 do not see the NaN either, checked below
        rest[1, :100] = False
        assert torch.equal(got[n][rest.cuda()], clean[n][rest.cuda()]), n
        close(got[n][0, 250:], (exp[n][0][0, 250:], exp[n][1][0, 250:]), n)
        assert torch.equal(got[n][0, :100], clean[n][0, :100]), n
        assert torch.isnan(got[n][0, 100:173]).any(), n
    assert torch.equal(got["h_last"], clean["h_last"])


def test_gates_at_their_ends():
    """Shut and open gates, rates of zero: the state is held, dropped, taken over."""
    inf = float("inf")
    t = make(1, 6, 8, "f32", h0=True, seed=2)
    t["ga"][0, :, 0], t["ga"][0, :, 1], t["gx"][0, :, 2], t["gx"][0, :, 3] = -inf, inf, -inf, inf
    t["ga"][0, :, 4] = torch.finfo(torch.float32).min
    t["gx"][0, :, 5] = torch.finfo(torch.float32).max
    t["rate"][6] = 0.0
    t["rate"][7] = 1e30
    t["ga"][0, :, 7] = 1.0
    got = run(t)
    h0 = t["h0"][0]
    for c in (0, 4, 6):      # held: a = 1, n = 0, and no slope
        assert torch.equal(got["h"][0, :, c], h0[c].expand(6)), c
        for n in ("dx", "dgate_a", "dgate_x"):
            assert torch.count_nonzero(got[n][0, :, c]) == 0, (n, c)
    # a shut gate hides its rate; a rate of zero still moves a (drate = -sum G a h r), if not the root
    assert got["drate"][0] == 0 and got["drate"][4] == 0
    u = torch.sigmoid(t["gx"][0, :, 7]) * t["x"][0, :, 7]
    assert torch.allclose(got["h"][0, :, 7], u, rtol=1e-6, atol=0)      # nothing is kept
    assert torch.isfinite(got["h"]).all() and all(torch.isfinite(a).all() for a in got.values())
    exp = want(dict(t, ga=t["ga"].clamp(-1e4, 1e4), gx=t["gx"].clamp(-1e4, 1e4)))
    close(got["drate"][6], (exp["drate"][0][6], exp["drate"][1][6]), "drate")
    for c in (1, 2, 3, 5):
        for n in ("h", "dx", "dgate_x"):
            v, b = exp[n][0][0, :, c], exp[n][1][0, :, c]
            close(got[n][0, :, c], (v, np.minimum(b, 1e-5 * (1 + np.abs(v)))), (n, c))


def test_a_channel_that_forgets_slowly_keeps_its_digits():
    """1 - a and 1 - a^2 near one: with the same gate at every token h is the geometric sum, and a in 32 bits alone
    would be off by 2^-25 / (1 - a) of it after all."""
    L, C = 700, 8
    t = make(1, L, C, "f32", gated=False, seed=4)
    t["rate"] = torch.full((C,), 1e-6, device="cuda")
    t["ga"].zero_()
    t["x"].fill_(1.0)
    got = host(run(t)["h"])[0, :, 0]
    rate = float(t["rate"][0])
    a = np.exp(-0.5 * rate)
    exp = np.sqrt(-np.expm1(-rate)) * (1 - a ** np.arange(1, L + 1)) / -np.expm1(-0.5 * rate)
    # per token one rounding of the state and one of a, both of 2^-24, and the root's 16 roundings
    assert (np.abs(got - exp) <= (2 * np.arange(1, L + 1) + 24) * ref.U * exp).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("B,C", [(1, 1), (8, 2048), (3, 330), (40, 2048), (5, 7)])
@pytest.mark.parametrize("gated,normalize", [(True, True), (False, False)])
def test_step(B, C, gated, normalize, kind):
    t = make(B, 1, C, kind, gated=gated, h0=True, seed=B + C)
    x, ga = t["x"][:, 0].contiguous(), t["ga"][:, 0].contiguous()
    gx = t["gx"][:, 0].contiguous() if gated else None
    exp = want(t, normalize)
    state = t["h0"].clone()
    h = api.s5_gated_scan_step(x, ga, gx, t["rate"], state, normalize=normalize)
    close(state, exp["h_last"], "state")
    close(h, (exp["h"][0][:, 0], exp["h"][1][:, 0]), "h")
    again = t["h0"].clone()
    assert api.s5_gated_scan_step(x, ga, gx, t["rate"], again, normalize=normalize, h=x) is x     # in place of x
    assert torch.equal(x, h) and torch.equal(again, state)


@pytest.mark.parametrize("kind", TYPES)
def test_parts_of_a_sequence_are_the_whole(kind):
    """Two calls with the state handed on, then single tokens; gradients through both calls."""
    t = make(2, 260, 48, kind, h0=True, seed=6)
    exp, cut = want(t), 131
    a = {n: v[:, :cut].contiguous() if v is not None and v.dim() == 3 else v for n, v in t.items()}
    b = {n: v[:, cut:].contiguous() if v is not None and v.dim() == 3 else v for n, v in t.items()}
    sa, sb = api.new_gated_scan_saved(a["x"]), api.new_gated_scan_saved(b["x"])
    ha, mid = api.s5_gated_scan_forward(a["x"], a["ga"], a["gx"], a["rate"], h0=t["h0"], h_last=True, saved=sa)
    state = mid.clone()
    hb, last = api.s5_gated_scan_forward(b["x"], b["ga"], b["gx"], b["rate"], h0=state, h_last=state, saved=sb)
    assert last is state                 # in place
    close(torch.cat([ha, hb], 1), exp["h"], "h")
    close(last, exp["h_last"], "h_last")
    gb = api.s5_gated_scan_backward(b["x"], b["ga"], b["gx"], b["rate"], b["dh"], sb, h0=mid, dh_last=t["dh_last"])
    ga = api.s5_gated_scan_backward(a["x"], a["ga"], a["gx"], a["rate"], a["dh"], sa, h0=t["h0"], dh_last=gb["dh0"])
    for n in ("dx", "dgate_a", "dgate_x"):
        close(torch.cat([ga[n], gb[n]], 1), exp[n], n)
    close(ga["dh0"], exp["dh0"], "dh0")
    state = mid.clone()
    for i in range(4):
        h = api.s5_gated_scan_step(*(b[n][:, i].contiguous() for n in ("x", "ga", "gx")), t["rate"], state)
        close(h, (exp["h"][0][:, cut + i], exp["h"][1][:, cut + i]), "token %d" % i)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("C,gap", [(64, 32), (40, 2), (40, 1)])
def test_views_of_a_fused_projection(C, gap, kind):
    t = make(2, 150, C, kind, h0=True, seed=8)
    fused = torch.full((2, 150, 4 * C + gap), float("nan"), device="cuda", dtype=TYPES[kind])
    v = dict(t)
    for i, n in enumerate(("x", "ga", "gx", "dh")):
        v[n] = fused[..., i * C:(i + 1) * C]
        v[n].copy_(t[n])
    assert same(run(v), run(t)) or (C + gap) % 8 != 0      # another vector width sums in another order
    exp, got = want(t), run(v)
    for n, e in exp.items():
        close(got[n], e, n)
    wide = torch.full((2, 150, C + 16), 7.0, device="cuda", dtype=TYPES[kind])
    h = api.s5_gated_scan_forward(v["x"], v["ga"], v["gx"], v["rate"], h0=t["h0"], h=wide[..., :C])
    close(h, exp["h"], "h")
    assert (wide[..., C:] == 7.0).all()


def test_empty_calls():
    for B, L in ((0, 5), (2, 0)):
        t = make(B, L, 8, "bf16", h0=True, seed=1)
        got = run(t)
        assert got["h"].shape == (B, L, 8) and torch.equal(got["h_last"], t["h0"]) and torch.equal(got["dh0"], t["dh_last"])
        assert torch.count_nonzero(got["drate"]) == 0
    t = make(2, 0, 8, "bf16", seed=1)
    assert torch.count_nonzero(run(t)["h_last"]) == 0
    assert api.s5_gated_scan_step(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, device="cuda"), None, torch.ones(8, device="cuda"),
                                  torch.empty(0, 8, device="cuda")).shape == (0, 8)


def test_equal_inputs_give_equal_bits():
    t = make(2, 3000, 128, "bf16", marks=0.01, seed=11)
    first = run(t)
    for _ in range(5):
        assert same(run(t), first)


def test_offsets_past_32_bits():
    """Rows 2^31 values apart and more: the last tokens of a long pitch."""
    L, C, ld = 70_000, 8, 32_000
    big = torch.empty(L * ld, device="cuda", dtype=torch.bfloat16)
    assert big.numel() > 1 << 31
    x = big.as_strided((1, L, C), (L * ld, ld, 1))
    t = make(1, L, C, "bf16", gated=False, seed=12)
    x.copy_(t["x"])
    h = api.s5_gated_scan_forward(x, t["ga"], None, t["rate"])
    assert torch.equal(h, api.s5_gated_scan_forward(t["x"], t["ga"], None, t["rate"]))
    out = big.as_strided((1, L, C), (L * ld, ld, 1), C)
    api.s5_gated_scan_forward(x, t["ga"], None, t["rate"], h=out)
    assert torch.equal(out, h)
