"""GPU tests of layer norm of a sum against float64, value by value (tests/_recurrent_ref.py derives the bounds)."""
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


def make(N, H, kind, weight=True, bias=True, residual=True, seed=0, mean=0.3):
    x = rnd((N, H), kind, seed + 1)[0] + mean
    return dict(x=x, r=rnd((N, H), kind, seed + 2)[0] if residual else None, w=rnd((H,), "f32", seed + 3)[0] if weight else None,
                b=rnd((H,), "f32", seed + 4)[0] if bias else None, dy=rnd((N, H), kind, seed + 5)[0],
                dt=rnd((N, H), kind, seed + 6)[0] if residual else None)


def run(t, eps=1e-5):
    saved = api.new_layernorm_saved(t["x"])
    out = api.s5_add_layernorm(t["x"], weight=t["w"], bias=t["b"], residual=t["r"], eps=eps, saved=saved)
    y, total = (out, t["x"]) if t["r"] is None else out
    g = api.s5_add_layernorm_backward(t["x"], t["dy"], saved, weight=t["w"], bias=t["b"], residual=t["r"], dtotal=t["dt"])
    return dict(g, y=y, total=total, saved=saved)


def check(t, eps=1e-5):
    got = run(t, eps)
    v = {n: host(a) for n, a in t.items()}
    exp = ref.norm(v["x"], v["w"], v["b"], v["r"], eps)
    close(got["y"], exp["y"], "y")
    close(got["total"], exp["total"], "total")
    close(got["saved"][:, 0], exp["mean"], "mean")
    close(got["saved"][:, 1], exp["inv"], "inv")
    s = host(got["saved"])
    exp = ref.norm_backward(exp["total"][0], v["dy"], s[:, 0], s[:, 1], v["w"], v["dt"])
    close(got["dx"], exp["dx"], "dx")
    for n, there in (("dweight", t["w"]), ("dbias", t["b"])):
        assert (got[n] is None) == (there is None)
        if there is not None:
            close(got[n], exp[n], n)


# one warp a row and several, vectors of every width, rows that fill no warp, the widest
WIDTHS = [1, 2, 7, 8, 64, 100, 255, 512, 513, 770, 1024, 2048, 2050, 2560, 4104, 8192, 8200, 16384, 16383, 12000]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, residual, kind):
    check(make(5, H, kind, residual=residual, seed=H))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [48, 770, 2048, 8192])
@pytest.mark.parametrize("N", [1, 37, 1500, 5000])
def test_rows(N, H, kind):
    if N * H > 4_000_000:
        N = 4_000_000 // H
    check(make(N, H, kind, seed=N + H))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
def test_without_weight_or_bias(weight, bias, kind):
    check(make(40, 264, kind, weight=weight, bias=bias, seed=3))


@pytest.mark.parametrize("H", [96, 2048, 4100])
def test_rows_far_from_zero_keep_their_digits(H):
    """Values of 1000 and a spread of 1: the sum of squares alone would lose six digits."""
    check(make(20, H, "f32", residual=False, seed=5, mean=1000.0))


def test_rows_of_one_value():
    """No spread: y is the bias, with eps as the only size."""
    t = make(4, 200, "f32", residual=False, seed=6)
    t["x"][:] = torch.tensor([0.0, 1.0, -3.0, 2.0 ** 20], device="cuda")[:, None]
    got = run(t)
    assert torch.equal(got["y"], t["b"].expand(4, 200))
    assert torch.isfinite(got["dx"]).all() and torch.equal(got["saved"][:, 0], t["x"][:, 0])


def test_a_bad_row_stays_alone():
    t = make(9, 512, "bf16", seed=7)
    clean = run(t)
    t["x"][4, 100] = float("nan")
    t["x"][6, 3] = float("inf")
    got = run(t)
    rest = torch.tensor([i not in (4, 6) for i in range(9)], device="cuda")
    for n in ("y", "total", "dx"):
        assert torch.equal(got[n][rest], clean[n][rest]), n
    assert torch.isnan(got["y"][4]).all() and torch.isnan(got["y"][6]).any()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [64, 770, 4096])
def test_in_place(H, kind):
    t = make(33, H, kind, seed=8)
    want = run(t)
    for which in ("x", "r"):
        u = {n: None if a is None else a.clone() for n, a in t.items()}
        y, total = api.s5_add_layernorm(u["x"], u["w"], u["b"], u["r"], total=u[which])
        assert total is u[which] and same(y, want["y"]) and same(total, want["total"])
        u = {n: None if a is None else a.clone() for n, a in t.items()}
        y, total = api.s5_add_layernorm(u["x"], u["w"], u["b"], u["r"], y=u[which])
        assert y is u[which] and same(y, want["y"]) and same(total, want["total"])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H,gap", [(64, 32), (40, 2), (40, 1), (4096, 8)])
def test_views(H, gap, kind):
    t = make(30, H, kind, seed=9)
    v = dict(t)
    for n in ("x", "r", "dy", "dt"):
        wide = torch.full((30, H + gap), float("nan"), device="cuda", dtype=TYPES[kind])
        v[n] = wide[:, :H]
        v[n].copy_(t[n])
    check(v)
    out = torch.full((30, H + 8), 7.0, device="cuda", dtype=TYPES[kind])
    y, _ = api.s5_add_layernorm(v["x"], v["w"], v["b"], v["r"], y=out[:, :H])
    assert (out[:, H:] == 7.0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [64, 770, 4096])
def test_backward_from_the_total_and_in_place(H, kind):
    """total for x and residual: the gradients are those of the rounded sum.  dx over any of its inputs."""
    t = make(33, H, kind, seed=13)
    saved = api.new_layernorm_saved(t["x"])
    _, total = api.s5_add_layernorm(t["x"], t["w"], t["b"], t["r"], saved=saved)
    got = api.s5_add_layernorm_backward(total, t["dy"], saved, t["w"], t["b"], dtotal=t["dt"])
    s = host(saved)
    exp = ref.norm_backward(host(total), host(t["dy"]), s[:, 0], s[:, 1], host(t["w"]), host(t["dt"]))
    for n in ("dx", "dweight", "dbias"):
        close(got[n], exp[n], n)
    want, lib, st = run(t), api._native.lib(), torch.cuda.current_stream().cuda_stream
    work = torch.empty(api.s5_add_layernorm_workspace_size(H), dtype=torch.uint8, device="cuda")
    for which in ("x", "r", "dy", "dt"):
        u = {n: a.clone() for n, a in t.items()}
        dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        at = [a for n in ("x", "r", "dy", "dt") for a in (u[n].data_ptr(), H)]
        assert lib.s5_add_layernorm_backward(*at, kind == "bf16", u["w"].data_ptr(), saved.data_ptr(), 33, H, u[which].data_ptr(), H,
                                             dw.data_ptr(), db.data_ptr(), work.data_ptr(), work.numel(), st) == 0
        assert same(u[which], want["dx"]) and same(dw, want["dweight"]) and same(db, want["dbias"])


def test_leading_axes_and_empty_calls():
    t = make(24, 64, "bf16", seed=10)
    y, total = api.s5_add_layernorm(t["x"].view(2, 3, 4, 64), t["w"], t["b"], t["r"].view(2, 3, 4, 64))
    assert same(y.view(24, 64), run(t)["y"]) and total.shape == (2, 3, 4, 64)
    one = api.s5_add_layernorm(t["x"][0], t["w"], t["b"])
    assert one.shape == (64,)
    e = make(0, 64, "bf16", seed=1)
    got = run(e)
    assert got["y"].shape == (0, 64) and torch.count_nonzero(got["dweight"]) == 0 and torch.count_nonzero(got["dbias"]) == 0


def test_equal_inputs_give_equal_bits():
    t = make(3000, 520, "bf16", seed=11)
    first = run(t)
    for _ in range(5):
        assert same(run(t), first)


def test_offsets_past_32_bits():
    N, H, ld = 70_000, 64, 32_000
    big = torch.empty(N * ld, device="cuda", dtype=torch.bfloat16)
    t = make(N, H, "bf16", seed=12)
    x = big.as_strided((N, H), (ld, 1))
    x.copy_(t["x"])
    assert same(run(dict(t, x=x)), run(t))


# several rows a block where the weights' gradients are summed in shared memory, and on both sides of where that begins
WIDE = [6144, 6145, 6148, 7001, 7002, 8191, 8192, 8193, 8200, 12289, 12290, 16384]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", WIDE)
def test_wide_rows_add_up(H, kind):
    t = make(500, H, kind, residual=H % 4 != 1, seed=H + 1)
    check(t)
    first = run(t)
    assert same(run(t), first)
    only = dict(t, w=None, b=None)
    assert run(only)["dweight"] is None
    check(only)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("H", [7001, 12000, 12290])
def test_wide_rows_in_place(H, kind):
    t = make(320, H, kind, seed=H + 2)
    want, lib, st = run(t), api._native.lib(), torch.cuda.current_stream().cuda_stream
    work = torch.empty(api.s5_add_layernorm_workspace_size(H), dtype=torch.uint8, device="cuda")
    for which in ("x", "r", "dy", "dt"):
        u = {n: a.clone() for n, a in t.items()}
        dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        at = [a for n in ("x", "r", "dy", "dt") for a in (u[n].data_ptr(), H)]
        assert lib.s5_add_layernorm_backward(*at, kind == "bf16", u["w"].data_ptr(), want["saved"].data_ptr(), 320, H,
                                             u[which].data_ptr(), H, dw.data_ptr(), db.data_ptr(), work.data_ptr(), work.numel(), st) == 0
        assert same(u[which], want["dx"]) and same(dw, want["dweight"]) and same(db, want["dbias"])
