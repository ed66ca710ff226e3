"""The parts of a gated recurrent block, as cases that can be timed and compared.

Three operators (include/s5.h has their definitions), each with its directions:

  scan, scan_train, scan_step   the gated linear recurrence h = a h + n u per channel: a
                                whole sequence, with its backward pass, one token
  conv, conv_train, conv_step   the short causal convolution of each channel along the
                                tokens: the same three
  norm, norm_train              layer norm of a sum of two rows, alone and with its
                                backward pass

run() computes them in plain torch operations in 32 bits where `own` is false,
and through diagonal_state_space_gb300.api where it is true.  exact() computes
them from their definitions in 64 bits: the recurrence token by token, the
convolution tap by tap, the norm from sums.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    scan = dict(op="scan", B=1, L=1, C=2048, type="bf16", gated=True, h0=False, packed=False, ragged=False)
    conv = dict(op="conv", B=1, L=1, C=2048, K=4, type="bf16", act="silu", bias=True, past=False, packed=False)
    norm = dict(op="norm", N=1, H=2048, type="bf16", residual=True)
    return [
        # the next token of a few users: the call's latency counts
        dict(scan, name="scan_step", op="scan_step", B=8),
        # one long document before generation starts: parallel along the tokens only
        dict(scan, name="scan_long", L=16384),
        # a training step over documents packed into rows, states start anew at each
        dict(scan, name="scan_train", op="scan_train", B=4, L=2048, C=2560, packed=True),
        # a small 32-bit run: odd channels, rows of their own lengths, a state carried in and out, no input gate
        dict(scan, name="scan_train_odd", op="scan_train", B=3, L=777, C=330, type="f32", gated=False, h0=True, ragged=True),
        # a full serving batch's next token, the last inputs of every sequence shifted on
        dict(conv, name="conv_step", op="conv_step", B=96, C=4096),
        # a batch of prompts that go on from cached inputs; the length ends inside a tile
        dict(conv, name="conv_prompt", B=8, L=1999, past=True),
        # a training step over packed documents
        dict(conv, name="conv_train", op="conv_train", B=4, L=2048, C=4096, packed=True),
        # a small 32-bit run: odd channels, three taps, no activation
        dict(conv, name="conv_train_odd", op="conv_train", B=2, L=501, C=331, K=3, type="f32", act=None, bias=False, past=True),
        # eight rows of a decode step
        dict(norm, name="norm_decode", N=8),
        # a training step's rows
        dict(norm, name="norm_train", op="norm_train", N=16384),
        # a small 32-bit run with an odd width
        dict(norm, name="norm_train_odd", op="norm_train", N=1237, H=770, type="f32", residual=False),
        # a prompt of a wide model
        dict(norm, name="norm_wide", N=4099, H=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "conv", "conv_train", "conv_step", "norm",
                     "norm_train", "norm_train"])
    case = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
    part = 1 if case["type"] == "bf16" else 2
    flag = lambda p=0.5: rng.random() < p  # noqa: E731
    if op.startswith("norm"):
        case["H"] = _log(rng, 64, 8192) if flag() else 128 * _log(rng, 1, 64)
        case["N"] = _log(rng, 1, max(1, 32_000_000 // part // case["H"]))
        case["residual"] = flag(0.7)
        return case
    case["C"] = 64 * _log(rng, 1, 64) if flag(0.7) else _log(rng, 1, 4096)
    if op.endswith("step"):
        case.update(B=_log(rng, 1, 128), L=1)
    else:
        values = (32_000_000 if not op.endswith("train") else 20_000_000) // part
        case["L"] = _log(rng, 1, min(16384, max(1, values // case["C"])))
        case["B"] = _log(rng, 1, max(1, min(16, values // (case["C"] * case["L"]))))
    many = case["L"] > 1
    if op.startswith("scan"):
        case.update(gated=flag(0.7), h0=flag() and not op.endswith("step"), packed=many and flag(0.4), ragged=many and flag(0.3))
    else:
        case.update(K=rng.choice([2, 3, 4, 4, 4, 5, 7, 8]), act=rng.choice(["silu", "silu", None]), bias=flag(),
                    past=flag() and not op.endswith("step"), packed=many and flag(0.4))
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    dt, op = _TYPES[case["type"]], case["op"]
    st = dict(case=dict(case))
    if op.startswith("norm"):
        N, H = case["N"], case["H"]
        # rows with a mean and a size of their own, as a residual stream has
        st["x"] = (rnd(N, H) + 0.3 * rnd(N, 1)).to(dt)
        st["residual"] = (rnd(N, H) * (1 + uni(N, 1))).to(dt) if case["residual"] else None
        st["weight"], st["bias"], st["eps"] = 1 + 0.2 * rnd(H), 0.1 * rnd(H), 1e-5
        if op == "norm_train":
            st["dy"] = rnd(N, H).to(dt)
            st["dtotal"] = rnd(N, H).to(dt) if case["residual"] else None
        return st
    B, L, C = case["B"], case["L"], case["C"]
    tok = (B, C) if op.endswith("step") else (B, L, C)
    st["x"] = rnd(*tok).to(dt)
    # documents of a few hundred tokens; the row's first token is one's first as well
    st["reset"] = torch.cat([torch.ones(B, 1, device=dev), uni(B, L - 1) < 1 / 400], 1).to(torch.bool) if case["packed"] else None
    if op.startswith("scan"):
        st["gate_a"] = rnd(*tok).to(dt)
        st["gate_x"] = rnd(*tok).to(dt) if case["gated"] else None
        # channels forget within one token to a few thousand
        st["rate"] = torch.exp(math.log(1e-3) + math.log(4e3) * uni(C))
        if op == "scan_step":
            st["state"] = rnd(B, C)
        else:
            st["h0"] = rnd(B, C) if case["h0"] else None
            st["lengths"] = (torch.ceil(uni(B) * L)).to(torch.int32) if case["ragged"] else None
        if op == "scan_train":
            st["dh"] = rnd(*tok).to(dt)
            st["dh_last"] = rnd(B, C) if case["h0"] else None
        return st
    K = case["K"]
    st["weight"] = rnd(C, K) * K ** -0.5
    st["bias"] = 0.1 * rnd(C) if case["bias"] else None
    if op == "conv_step":
        st["state"] = rnd(B, K - 1, C).to(dt)
    else:
        st["past"] = rnd(B, K - 1, C).to(dt) if case["past"] else None
    if op == "conv_train":
        st["dy"] = rnd(*tok).to(dt)
    return st


# ------------------------------------------------------------------ plain forms
def _pair_scan(a, e):
    """All prefixes of h = a h + e along axis 1, by doubling: pairs (a, e) of 1, 2, 4, ... tokens are joined."""
    n = 1
    while n < a.shape[1]:
        e = torch.cat([e[:, :n], e[:, n:] + a[:, n:] * e[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return a, e


def _valid(st, L):
    """[B,L,1] truth values: which tokens belong to their row."""
    if st["lengths"] is None:
        return None
    return (torch.arange(L, device=st["x"].device) < st["lengths"][:, None])[..., None]


def _gates(st):
    """log decay without its rate, and the input gate: both sigmoids, in 32 bits."""
    r = 1 / (1 + torch.exp(-st["gate_a"].float()))
    s = 1 / (1 + torch.exp(-st["gate_x"].float())) if st["gate_x"] is not None else torch.ones_like(r)
    return r, s


def _plain_scan(st):
    case, dt = st["case"], _TYPES[st["case"]["type"]]
    r, s = _gates(st)
    la = -st["rate"] * r
    a, n = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    x = st["x"].float()
    if case["op"] == "scan_step":
        st["state"].mul_(a).add_(n * s * x)
        return dict(h=st["state"].to(dt), state=st["state"])
    B, L, C = x.shape
    valid = _valid(st, L)
    if st["reset"] is not None:
        a, n = torch.where(st["reset"][..., None], 0.0, a), torch.where(st["reset"][..., None], 1.0, n)
    u = s * x
    e = n * u
    if valid is not None:                # tokens past the end leave the state as it is
        a, e = torch.where(valid, a, 1.0), torch.where(valid, e, 0.0)
    h0 = st["h0"] if st["h0"] is not None else torch.zeros(B, C, device=x.device)
    run, h = _pair_scan(a, e)
    h = h + run * h0[:, None]
    out = dict(h=h, h_last=h[:, -1].clone())
    if valid is not None:
        out["h"] = torch.where(valid, h, 0.0)
    if case["op"] == "scan_train":
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        g = st["dh"].float()
        if valid is not None:
            g = torch.where(valid, g, 0.0)
        if st["dh_last"] is not None:
            g = torch.cat([g[:, :-1], g[:, -1:] + st["dh_last"][:, None]], 1)
        # from the end: G_t = g_t + a_{t+1} G_{t+1}
        later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        g = _pair_scan(later.flip(1), g.flip(1))[1].flip(1)
        root = torch.where(n > 0, a * a / n, 0.0) * u
        dla = g * (a * before - root)
        if valid is not None:
            dla = torch.where(valid, dla, 0.0)
        du = n * g if valid is None else torch.where(valid, n * g, 0.0)
        out.update(dx=(du * s), dgate_a=-st["rate"] * dla * r * (1 - r), drate=-(dla * r).sum((0, 1)))
        if st["gate_x"] is not None:
            out["dgate_x"] = du * x * s * (1 - s)
        if st["h0"] is not None:
            out["dh0"] = a[:, 0] * g[:, 0]
    return {k: v.to(dt) if k in ("h", "dx", "dgate_a", "dgate_x") else v for k, v in out.items()}


def _document(reset):
    """[B,L] which document a token is of, counted from the row's start (0: goes on from the past)."""
    return reset.long().cumsum(1)


def _window(st, x):
    """The K inputs of each token [B,L,K,C], zeros where they are another document's."""
    B, L, C = x.shape
    K = st["case"]["K"]
    before = st["past"].float() if st["past"] is not None else torch.zeros(B, K - 1, C, device=x.device)
    full = torch.cat([before, x], 1)
    w = torch.stack([full[:, j:j + L] for j in range(K)], 2)
    if st["reset"] is not None:
        doc = torch.cat([torch.zeros(B, K - 1, dtype=torch.long, device=x.device), _document(st["reset"])], 1)
        same = torch.stack([doc[:, j:j + L] == doc[:, K - 1:] for j in range(K)], 2)
        w = torch.where(same[..., None], w, 0.0)
    return full, w


def _plain_conv(st):
    case, dt = st["case"], _TYPES[st["case"]["type"]]
    K, w, x = case["K"], st["weight"], st["x"].float()
    b = st["bias"] if st["bias"] is not None else 0.0
    if case["op"] == "conv_step":
        seen = torch.cat([st["state"].float(), x[:, None]], 1)
        p = (seen * w.t()).sum(1) + b
        st["state"].copy_(seen[:, 1:])
        return dict(y=(p / (1 + torch.exp(-p)) if case["act"] else p).to(dt), state=st["state"])
    full, win = _window(st, x)
    p = (win * w.t()).sum(2) + b
    sig = 1 / (1 + torch.exp(-p))
    last = full[:, full.shape[1] - (K - 1):]
    if st["reset"] is not None:          # the next call sees nothing of an earlier document either
        doc = torch.cat([torch.zeros(x.shape[0], K - 1, dtype=torch.long, device=x.device), _document(st["reset"])], 1)
        last = torch.where((doc[:, doc.shape[1] - (K - 1):] == doc[:, -1:])[..., None], last, 0.0)
    out = dict(y=(p * sig if case["act"] else p).to(dt), past=last.to(dt))
    if case["op"] == "conv_train":
        dp = st["dy"].float()
        if case["act"]:
            dp = dp * sig * (1 + p * (1 - sig))
        dfull = torch.zeros_like(full)
        L = x.shape[1]
        for j in range(K):
            part = dp * w[:, j]
            if st["reset"] is not None:
                doc = torch.cat([torch.zeros(x.shape[0], K - 1, dtype=torch.long, device=x.device), _document(st["reset"])], 1)
                part = torch.where((doc[:, j:j + L] == doc[:, K - 1:])[..., None], part, 0.0)
            dfull[:, j:j + L] += part
        out.update(dx=dfull[:, K - 1:].to(dt), dweight=(win * dp[:, :, None]).sum((0, 1)).t().contiguous())
        if st["bias"] is not None:
            out["dbias"] = dp.sum((0, 1))
        if st["past"] is not None:
            out["dpast"] = dfull[:, :K - 1].to(dt)
    return out


def _plain_norm(st):
    case, dt = st["case"], _TYPES[st["case"]["type"]]
    s = st["x"].float()
    if case["residual"]:
        s = s + st["residual"].float()
    c = s - s.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + st["eps"])
    n = c * r
    out = dict(y=(n * st["weight"] + st["bias"]).to(dt))
    if case["residual"]:
        out["total"] = s.to(dt)
    if case["op"] == "norm_train":
        dy = st["dy"].float()
        g = dy * st["weight"]
        dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
        if case["residual"]:
            dx = dx + st["dtotal"].float()
        out.update(dx=dx.to(dt), dweight=(dy * n).sum(0), dbias=dy.sum(0))
    return out


def _plain(st):
    kind = st["case"]["op"].split("_")[0]
    return dict(scan=_plain_scan, conv=_plain_conv, norm=_plain_norm)[kind](st)


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    from diagonal_state_space_gb300 import api
    case, op = st["case"], st["case"]["op"]
    there = lambda d: {n: t for n, t in d.items() if t is not None}  # noqa: E731
    if op == "scan_step":
        return dict(h=api.s5_gated_scan_step(st["x"], st["gate_a"], st["gate_x"], st["rate"], st["state"]), state=st["state"])
    if op.startswith("scan"):
        four = (st["x"], st["gate_a"], st["gate_x"], st["rate"])
        rows = dict(h0=st["h0"], reset=st["reset"], lengths=st["lengths"])
        saved = api.new_gated_scan_saved(st["x"]) if op == "scan_train" else None
        h, last = api.s5_gated_scan_forward(*four, h_last=True, saved=saved, **rows)
        out = dict(h=h, h_last=last)
        if op == "scan_train":
            out.update(there(api.s5_gated_scan_backward(*four, st["dh"], saved, dh_last=st["dh_last"], **rows)))
        return out
    if op == "conv_step":
        y = api.s5_short_conv_step(st["x"], st["weight"], st["state"], bias=st["bias"], activation=case["act"])
        return dict(y=y, state=st["state"])
    if op.startswith("conv"):
        kw = dict(bias=st["bias"], activation=case["act"], past=st["past"], reset=st["reset"])
        y, past = api.s5_short_conv_forward(st["x"], st["weight"], past_out=True, **kw)
        out = dict(y=y, past=past)
        if op == "conv_train":
            out.update(there(api.s5_short_conv_backward(st["x"], st["weight"], st["dy"], **kw)))
        return out
    saved = api.new_layernorm_saved(st["x"]) if op == "norm_train" else None
    kw = dict(weight=st["weight"], bias=st["bias"])
    y = api.s5_add_layernorm(st["x"], residual=st["residual"], eps=st["eps"], saved=saved, **kw)
    out, total = dict(y=y), st["x"]
    if case["residual"]:
        out["y"], total = y
        out["total"] = total
    if op == "norm_train":
        out.update(there(api.s5_add_layernorm_backward(st["x"], st["dy"], saved, residual=st["residual"], dtotal=st["dtotal"], **kw)))
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, op = _TYPES[case["type"]].itemsize, case["op"]
    if op.startswith("norm"):
        n, H, two = case["N"] * case["H"], case["H"], 2 if case["residual"] else 1
        if op == "norm":
            return dict(bytes=2 * two * e * n + 8 * H, flops=8 * n)
        # x, dy and the residual's pair in, y, total and dx out
        return dict(bytes=(3 * two + (1 if two == 1 else 0)) * e * n + 16 * H, flops=22 * n)
    B, L, C = case["B"], case["L"], case["C"]
    n = B * L * C
    marks = B * L if case["packed"] else 0
    if op.startswith("scan"):
        ins, ends = 3 if case["gated"] else 2, 4 * B * C * (2 if case["h0"] else 1)
        if op == "scan_step":
            return dict(bytes=(ins + 1) * e * n + 8 * n + 4 * C, flops=16 * n)
        if op == "scan":
            return dict(bytes=(ins + 1) * e * n + marks + ends + 4 * C, flops=16 * n)
        return dict(bytes=2 * (ins + 1) * e * n + marks + 2 * ends + 8 * C, flops=44 * n)
    K = case["K"]
    taps = 4 * C * (K + (1 if case["bias"] else 0))
    if op == "conv_step":
        return dict(bytes=2 * e * n + 2 * e * (K - 1) * n + taps, flops=(2 * K + 5) * n)
    ends = e * B * (K - 1) * C * (2 if case["past"] else 1)
    if op == "conv":
        return dict(bytes=2 * e * n + marks + ends + taps, flops=(2 * K + 5) * n)
    return dict(bytes=4 * e * n + marks + ends + 2 * taps + (e * B * (K - 1) * C if case["past"] else 0),
                flops=(8 * K + 15) * n)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_scan(st):
    case = st["case"]
    rate = st["rate"].double()
    sg = torch.sigmoid(st["gate_a"].double())
    x = st["x"].double()
    open_ = torch.sigmoid(st["gate_x"].double()) if st["gate_x"] is not None else None
    v = x if open_ is None else open_ * x
    decay = (-rate * sg).exp()
    gain = (-(-2 * rate * sg).expm1()).sqrt()
    if case["op"] == "scan_step":
        h = decay * st["state"].double() + gain * v
        return dict(h=h, state=h)
    B, L, C = x.shape
    ends = [L] * B if st["lengths"] is None else st["lengths"].tolist()
    fresh = st["reset"]
    if fresh is not None:
        decay = decay.masked_fill(fresh[..., None], 0.0)
        gain = gain.masked_fill(fresh[..., None], 1.0)
    live = torch.tensor([[float(t < n) for n in ends] for t in range(L)], dtype=torch.float64).to(x.device)[..., None]
    s = st["h0"].double() if st["h0"] is not None else torch.zeros(B, C, dtype=torch.float64, device=x.device)
    first, h = s, torch.empty_like(x)
    whole = st["lengths"] is None
    push = gain * v
    for t in range(L):
        new = torch.addcmul(push[:, t], decay[:, t], s)
        s = new if whole else torch.lerp(s, new, live[t])
        h[:, t] = s
    out = dict(h=h if whole else h * live.transpose(0, 1), h_last=s)
    if case["op"] == "scan":
        return out
    dh = st["dh"].double()
    z = st["dh_last"].double() if st["dh_last"] is not None else torch.zeros_like(s)
    G = torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        at = z + dh[:, t]
        G[:, t] = at if whole else at * live[t]
        z = decay[:, t] * at if whole else torch.lerp(z, decay[:, t] * at, live[t])
    prev = torch.roll(h, 1, 1)
    prev[:, 0] = first
    slope = (decay ** 2 / gain).masked_fill(gain == 0, 0.0)
    by_log = G * (decay * prev - slope * v)
    by_gate = -by_log * sg
    out.update(drate=by_gate.sum((0, 1)), dgate_a=rate * by_gate * (1 - sg))
    into = G * gain
    out["dx"] = into if open_ is None else into * open_
    if open_ is not None:
        out["dgate_x"] = into * x * open_ * (1 - open_)
    if st["h0"] is not None:
        out["dh0"] = z
    return out


def _exact_conv(st):
    case = st["case"]
    K, w = case["K"], st["weight"].double()
    add = st["bias"].double() if st["bias"] is not None else torch.zeros(case["C"], dtype=torch.float64, device=w.device)
    if case["op"] == "conv_step":
        x, old = st["x"].double(), st["state"].double()
        p = add + w[:, K - 1] * x
        for j in range(K - 1):
            p = p + w[:, j] * old[:, j]
        state = torch.cat([old[:, 1:], x[:, None]], 1)
        return dict(y=p * torch.sigmoid(p) if case["act"] else p, state=state)
    x = st["x"].double()
    B, L, C = x.shape
    # tokens since the document began; the tap `back` tokens ago counts where there are as many.  A row that no
    # reset opens goes on from its past.
    age = torch.full((B, L), K, dtype=torch.long, device=x.device)
    if st["reset"] is not None:
        t = torch.arange(L, device=x.device).expand(B, L)
        began = torch.where(st["reset"], t, -1).cummax(1).values
        age = torch.where(began >= 0, t - began, K)
    past = st["past"].double() if st["past"] is not None else torch.zeros(B, K - 1, C, dtype=torch.float64, device=x.device)
    line = torch.cat([past, x], 1)
    p = add.expand(B, L, C).clone()
    for back in range(K):
        tap = line[:, K - 1 - back:K - 1 - back + L]
        p += w[:, K - 1 - back] * tap * (age >= back)[..., None]
    sig = torch.sigmoid(p)
    seen = age[:, -1:] >= torch.arange(K - 2, -1, -1, device=x.device)
    out = dict(y=p * sig if case["act"] else p, past=line[:, L:] * seen[..., None])
    if case["op"] == "conv":
        return out
    dp = st["dy"].double()
    if case["act"]:
        dp = dp * (sig + p * sig * (1 - sig))
    dline, dw = torch.zeros_like(line), torch.zeros_like(w)
    for back in range(K):
        at, j = slice(K - 1 - back, K - 1 - back + L), K - 1 - back
        d = dp * (age >= back)[..., None]
        dw[:, j] = (d * line[:, at]).sum((0, 1))
        dline[:, at] += d * w[:, j]
    out.update(dx=dline[:, K - 1:], dweight=dw)
    if st["bias"] is not None:
        out["dbias"] = dp.sum((0, 1))
    if st["past"] is not None:
        out["dpast"] = dline[:, :K - 1]
    return out


def _exact_norm(st):
    case = st["case"]
    s = st["x"].double()
    if st["residual"] is not None:
        s = s + st["residual"].double()
    H = case["H"]
    mean = s.sum(-1, keepdim=True) / H
    var = ((s - mean) ** 2).sum(-1, keepdim=True) / H
    inv = (var + st["eps"]) ** -0.5
    w = st["weight"].double()
    out = dict(y=torch.addcmul(st["bias"].double(), (s - mean) * inv, w))
    if st["residual"] is not None:
        out["total"] = s
    if case["op"] == "norm_train":
        dy = st["dy"].double()
        out["dweight"], out["dbias"] = (dy * (s - mean) * inv).sum(0), dy.sum(0)
        # through the row's mean and size one after the other
        dc = dy * w * inv
        dvar = -0.5 * inv ** 3 * (dy * w * (s - mean)).sum(-1, keepdim=True)
        dc = dc + 2 * dvar * (s - mean) / H
        out["dx"] = dc - dc.sum(-1, keepdim=True) / H
        if st["dtotal"] is not None:
            out["dx"] = out["dx"] + st["dtotal"].double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return dict(scan=_exact_scan, conv=_exact_conv, norm=_exact_norm)[kind](st)
