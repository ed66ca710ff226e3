"""The sequence-mixer operators beside the S5 layer, as cases that can be timed and compared.

Four operators (include/s5.h has their definitions):

  step     one token of the gated delta rule per sequence, state updated in place
  prefill  the gated delta rule over whole sequences, with the state it ends in
  train    the same forward and its backward pass
  qk       norms of queries and keys for each head with the position rotation in
           the same pass, forward only or with its backward pass
  rotary   the position rotation alone

run() computes them in plain torch operations in 32 bits where `own` is false,
and through diagonal_state_space_gb300.api where it is true.  exact() computes
them from their definitions, token by token, in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ------------------------------------------------------------------ the cases
def listed():
    delta = dict(op="prefill", B=1, L=1, Hk=8, Hv=16, Dk=128, Dv=128, type="bf16", s0=False)
    qk = dict(op="qk", B=1, L=1, Hq=16, Hk=16, D=128, type="bf16", norm="rms", layout="half", rot=128,
              scaling="none", start=0, backward=False)
    rot = dict(op="rotary", B=1, L=1, H=16, D=128, type="bf16", layout="half", rot=128, scaling="none", start=0)
    return [
        # one user's next token: 1 MB of state, the call's latency counts
        dict(delta, name="step_one", op="step", B=1),
        # a full serving batch: every sequence's state is read and written (402 MB)
        dict(delta, name="step_batch", op="step", B=96, Hk=16, Hv=32),
        # one long document before generation starts: few heads, a long recurrence
        dict(delta, name="prefill_long", B=1, L=16384),
        # a batch of prompts continued from cached states; the length ends inside a chunk
        dict(delta, name="prefill_batch", B=8, L=1999, Hk=16, Hv=32, s0=True),
        # 32-bit model with odd head sizes and a group of three value heads to a key head
        dict(delta, name="prefill_odd", B=3, L=333, Hk=2, Hv=6, Dk=48, Dv=80, type="f32", s0=True),
        # a training step's mixer
        dict(delta, name="train_batch", op="train", B=4, L=2048),
        # a small 32-bit training run, ragged length, a state carried in and out
        dict(delta, name="train_small", op="train", B=2, L=500, Hk=4, Hv=4, Dk=64, Dv=64, type="f32", s0=True),
        # queries and keys of the next token of eight sequences, far into their contexts
        dict(qk, name="qk_decode", B=8, start=100_000),
        # a prompt's queries and keys: grouped heads, unit norms, half of the head rotated
        dict(qk, name="qk_prompt", B=2, L=8191, Hq=32, Hk=8, norm="l2", rot=64),
        # a training step's queries and keys with their learned weights' gradients
        dict(qk, name="qk_train", B=4, L=4096, backward=True),
        # a long context with interpolated frequencies, neighbouring pairs
        dict(rot, name="rotary_long", L=32768, H=32, layout="interleaved", scaling="by_parts", start=1_000_000),
        # 32-bit values, odd sizes, part of the head
        dict(rot, name="rotary_odd", B=3, L=517, H=5, D=80, type="f32", rot=48, scaling="ntk", start=77),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "prefill", "prefill", "train", "qk", "rotary"])
    if op in ("step", "prefill", "train"):
        half = rng.random() < 0.7
        Hk = rng.choice([2, 4, 8, 16])
        group = rng.choice([1, 2, 2, 3]) if Hk <= 8 else rng.choice([1, 2])
        Dk, Dv = rng.choice([(128, 128)] * 3 + [(64, 64), (64, 128), (128, 64)]) if half else (
            4 * rng.randint(8, 32), 4 * rng.randint(8, 32))
        case = dict(op=op, B=1, L=1, Hk=Hk, Hv=Hk * group, Dk=Dk, Dv=Dv, type="bf16" if half else "f32",
                    s0=op != "step" and rng.random() < 0.5)
        if op == "step":
            case["B"] = _log(rng, 1, 96)
            return case
        # tokens times heads stay below the largest listed case's
        tokens = (8 * 1999 * 32 if op == "prefill" else 4 * 2048 * 16) // (1 if half else 4)
        case["L"] = _log(rng, 3, min(tokens // case["Hv"], 16384 if op == "prefill" else 2048))
        case["B"] = _log(rng, 1, max(1, min(16, tokens // (case["L"] * case["Hv"]))))
        return case
    case = dict(op=op, B=1, L=1, type=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "ntk", "by_parts"]), start=_log(rng, 1, 1_000_000))
    case["D"] = rng.choice([64, 80, 96, 128, 128, 256])
    case["rot"] = rng.choice([case["D"], case["D"] // 2])
    if op == "rotary":
        case["H"] = heads = rng.randint(1, 32)
        passes = 2
    else:
        case["Hk"] = rng.choice([1, 2, 4, 8])
        case["Hq"] = case["Hk"] * rng.choice([1, 2, 4])
        case["norm"] = rng.choice(["rms", "l2"])
        case["backward"] = rng.random() < 0.5
        heads, passes = case["Hk"] + case["Hq"], 4 if case["backward"] else 2
    # at most 500 MB move
    tokens = 500_000_000 // (passes * heads * case["D"] * _TYPES[case["type"]].itemsize)
    case["L"] = _log(rng, 1, min(16384, tokens))
    case["B"] = _log(rng, 1, max(1, min(8, tokens // case["L"])))
    return case


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Angle per position of each rotated pair, and the factor on the rotated values, for a
    model trained on 8192 positions and used on eight times as many."""
    n, base, factor, trained = case["rot"] // 2, 10000.0, 8.0, 8192
    i = torch.arange(n, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base *= factor ** (2 * n / max(1, 2 * n - 2))
    freq = base ** (-i / n)
    if case["scaling"] == "linear":
        freq = freq / factor
    if case["scaling"] == "by_parts":
        turns = trained * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1 - keep)
        return freq, 0.1 * math.log(factor) + 1.0
    return freq, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    B, L, dt = case["B"], case["L"], _TYPES[case["type"]]
    st = dict(case=dict(case))
    if case["op"] in ("step", "prefill", "train"):
        Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        tok = (B,) if case["op"] == "step" else (B, L)
        # queries and keys come out of an activation with a positive mean and have unit norm
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
        for name, h, d in (("q", Hk, Dk), ("k", Hk, Dk)):
            x = rnd(*tok, h, d)
            st[name] = unit(x * torch.sigmoid(x)).to(dt)
        st["v"] = rnd(*tok, Hv, Dv).to(dt)
        # log decays -A softplus(x + b): A in [1, 16) per head, step sizes of 1e-3 to 1e-1
        A, step = 1 + 15 * uni(Hv), torch.exp(math.log(1e-3) + math.log(100.0) * uni(Hv))
        bias = step + torch.log(-torch.expm1(-step))
        st["g"] = -A * torch.nn.functional.softplus(rnd(*tok, Hv) + bias)
        st["beta"] = torch.sigmoid(rnd(*tok, Hv))
        st["scale"] = Dk ** -0.5
        if case["op"] == "step":
            st["state"] = rnd(B, Hv, Dk, Dv) * 0.2
        else:
            st["s0"] = rnd(B, Hv, Dk, Dv) * 0.2 if case["s0"] else None
        if case["op"] == "train":
            st["do"] = rnd(B, L, Hv, Dv).to(dt)
            st["ds_last"] = rnd(B, Hv, Dk, Dv) * 0.1 if case["s0"] else None
        return st
    freq, amp = _frequencies(case)
    st["freq"], st["amp"] = freq.to(dev), amp
    st["pos"] = (torch.arange(L, device=dev) + case["start"]).expand(B, L).contiguous()
    if case["op"] == "rotary":
        st["x"] = rnd(B, L, case["H"], case["D"]).to(dt)
        return st
    for name, h in (("q", case["Hq"]), ("k", case["Hk"])):
        st[name] = rnd(B, L, h, case["D"]).to(dt)
        st["d" + name] = rnd(B, L, h, case["D"]).to(dt) if case["backward"] else None
        st["w" + name] = 1 + 0.2 * rnd(case["D"]) if case["norm"] == "rms" else None
    st["eps"] = 1e-6
    return st


# ------------------------------------------------------------------ plain forms
def _inverse(a):
    """Inverse of unit lower-triangular 64 x 64 matrices, from diagonal blocks of 1, 2, 4, ... rows:
    [[A, 0], [C, B]]^-1 = [[A^-1, 0], [-B^-1 C A^-1, B^-1]]."""
    n, s = a.shape[-1], 1
    t = torch.ones(*a.shape[:-2], n, 1, 1, dtype=a.dtype, device=a.device)
    while s < n:
        blocks = a.reshape(*a.shape[:-2], n // (2 * s), 2 * s, n // (2 * s), 2 * s)
        own_block = torch.diagonal(blocks, dim1=-4, dim2=-2).movedim(-1, -3)
        low = own_block[..., s:, :s]
        t1, t2 = t[..., 0::2, :, :], t[..., 1::2, :, :]
        left = torch.cat([t1, -(t2 @ low @ t1)], dim=-2)
        right = torch.cat([torch.zeros_like(t2), t2], dim=-2)
        t, s = torch.cat([left, right], dim=-1), 2 * s
    return t[..., 0, :, :]


def _delta(q, k, v, g, beta, s0, scale):
    """The gated delta rule in chunks of 64 tokens, in 32 bits.  Returns o [B,L,Hv,Dv] and the last state."""
    (B, L, Hk, Dk), (Hv, Dv) = q.shape, v.shape[2:]
    pad = -L % _CHUNK
    N = (L + pad) // _CHUNK

    def chunks(x):  # [B,L,H,...] -> [N,B,Hv,64,...]
        x = torch.nn.functional.pad(x, [0, 0] * (x.dim() - 2) + [0, pad])
        x = x.reshape(B, N, _CHUNK, *x.shape[2:]).movedim(3, 1).movedim(2, 0)
        return x.repeat_interleave(Hv // x.shape[2], dim=2)

    q, k, v, g, beta = chunks(q) * scale, chunks(k), chunks(v), chunks(g), chunks(beta)
    G = g.double().cumsum(-1)  # differences of long sums
    i = torch.arange(_CHUNK, device=q.device)
    decay = torch.exp(torch.where(i[:, None] >= i, G[..., :, None] - G[..., None, :], -torch.inf)).float()
    up, down, last = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None], G[..., -1:].exp().float()[..., None]
    kk = (k @ k.mT) * decay * beta[..., None]
    a = torch.where(i[:, None] > i, kk, 0.0)
    t = _inverse(a) * beta[..., None, :]
    qk = (q @ k.mT) * decay
    kup, qup, kdown = k * up, q * up, (k * down).mT
    s = s0 if s0 is not None else torch.zeros(B, Hv, Dk, Dv, device=q.device)
    out = []
    for n in range(N):
        u = t[n] @ (v[n] - kup[n] @ s)
        out.append(qup[n] @ s + qk[n] @ u)
        s = last[n] * s + kdown[n] @ u
    o = torch.stack(out).movedim(0, 2).reshape(B, Hv, N * _CHUNK, Dv)[:, :, :L].transpose(1, 2)
    return o, s


def _rotate(x, cos, sin, layout):
    """Rotates pairs of the first 2 * cos.shape[-1] values of each head."""
    n = cos.shape[-1]
    a, b = (x[..., :n], x[..., n:2 * n]) if layout == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
    c, s = cos[..., None, :], sin[..., None, :]
    y = torch.cat([a * c - b * s, b * c + a * s], -1) if layout == "half" else torch.stack(
        [a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _norm(x, w, norm, eps):
    if norm == "rms":
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + eps)


def _plain(st):
    case, dt = st["case"], _TYPES[st["case"]["type"]]
    if case["op"] == "step":
        q, k, v = st["q"].float() * st["scale"], st["k"].float(), st["v"].float()
        group = case["Hv"] // case["Hk"]
        q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
        s = st["state"]
        s.mul_(torch.exp(st["g"])[..., None, None])
        u = st["beta"][..., None] * (v - (k[..., None] * s).sum(-2))
        s.add_(k[..., None] * u[..., None, :])
        return dict(o=(q[..., None] * s).sum(-2).to(dt), state=s)
    if case["op"] == "prefill":
        o, s = _delta(st["q"].float(), st["k"].float(), st["v"].float(), st["g"], st["beta"], st["s0"], st["scale"])
        return dict(o=o.to(dt), s_last=s)
    if case["op"] == "train":
        ins = [st[n].float().requires_grad_() if n != "s0" else st[n] for n in ("q", "k", "v", "g", "beta", "s0")]
        ins = [x.detach().requires_grad_() if x is not None else None for x in ins]
        o, s = _delta(*ins, st["scale"])
        outs, seeds = ([o, s], [st["do"].float(), st["ds_last"]]) if st["ds_last"] is not None else ([o], [st["do"].float()])
        names = [n for n, x in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), ins) if x is not None]
        grads = dict(zip(names, torch.autograd.grad(outs, [x for x in ins if x is not None], seeds)))
        return dict(grads, o=o.detach().to(dt), s_last=s.detach(),
                    **{n: grads[n].to(dt) for n in ("dq", "dk", "dv")})
    angle = st["pos"].double()[..., None] * st["freq"]
    cos, sin = (torch.cos(angle) * st["amp"]).float(), (torch.sin(angle) * st["amp"]).float()
    if case["op"] == "rotary":
        return _rotate(st["x"].float(), cos, sin, case["layout"]).to(dt)
    out = {}
    for n in ("q", "k"):
        x, w = st[n].float(), st["w" + n]
        if case["backward"]:
            x, w = x.requires_grad_(), None if w is None else w.detach().requires_grad_()
        y = _rotate(_norm(x, w, case["norm"], st["eps"]), cos, sin, case["layout"])
        out[n] = y.detach().to(dt)
        if case["backward"]:
            got = torch.autograd.grad(y, [x] if w is None else [x, w], st["d" + n].float())
            out["d" + n] = got[0].to(dt)
            if w is not None:
                out["dw" + n] = got[1]
    return out


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    from diagonal_state_space_gb300 import api
    case = st["case"]
    if case["op"] == "step":
        o = api.s5_delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], scale=st["scale"])
        return dict(o=o, state=st["state"])
    if case["op"] == "prefill":
        o, s = api.s5_delta_forward(st["q"], st["k"], st["v"], st["g"], st["beta"], scale=st["scale"], s0=st["s0"],
                                    s_last=True)
        return dict(o=o, s_last=s)
    if case["op"] == "train":
        saved = api.new_delta_saved(st["q"], st["v"])
        o, s = api.s5_delta_forward(st["q"], st["k"], st["v"], st["g"], st["beta"], scale=st["scale"], s0=st["s0"],
                                    s_last=True, saved=saved)
        grads = api.s5_delta_backward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"], saved,
                                      scale=st["scale"], s0=st["s0"], ds_last=st["ds_last"])
        return dict({n: x for n, x in grads.items() if x is not None}, o=o, s_last=s)
    rot = dict(layout=case["layout"], amplitude=st["amp"])
    if case["op"] == "rotary":
        return api.s5_rotary(st["x"], st["pos"], st["freq"], **rot)
    rot.update(norm=case["norm"], eps=st["eps"])
    q, k = api.s5_qk_norm_rotary(st["q"], st["k"], st["pos"], st["freq"], q_weight=st["wq"], k_weight=st["wk"], **rot)
    out = dict(q=q, k=k)
    if case["backward"]:
        g = api.s5_qk_norm_rotary_backward(st["q"], st["k"], st["dq"], st["dk"], st["pos"], st["freq"],
                                           q_weight=st["wq"], k_weight=st["wk"], **rot)
        out.update({n: x for n, x in g.items() if x is not None})
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, B, L = _TYPES[case["type"]].itemsize, case["B"], case["L"]
    if case["op"] in ("step", "prefill", "train"):
        Hk, Hv, Dk, Dv, T = case["Hk"], case["Hv"], case["Dk"], case["Dv"], B * L
        states = 4 * B * Hv * Dk * Dv
        qk, v, gates = 2 * e * T * Hk * Dk, e * T * Hv * Dv, 8 * T * Hv
        fwd = 6 * T * Hv * Dk * Dv  # k S, the outer product, q S
        if case["op"] == "step":
            return dict(bytes=2 * states + qk + 2 * v + gates, flops=fwd)
        ends = states * (2 if case["s0"] else 1)
        if case["op"] == "prefill":
            return dict(bytes=qk + 2 * v + gates + ends, flops=fwd)
        # backward: q dO, k dS, k dv, dS u, S dO, S dv products over the recomputed states
        return dict(bytes=2 * qk + 4 * v + 2 * gates + 2 * ends, flops=fwd + 14 * T * Hv * Dk * Dv)
    T, D = B * L, case["D"]
    if case["op"] == "rotary":
        return dict(bytes=2 * e * T * case["H"] * D + 8 * T, flops=3 * T * case["H"] * case["rot"])
    n = T * (case["Hq"] + case["Hk"]) * D
    weights = 8 * D if case["norm"] == "rms" else 0
    if case["backward"]:
        return dict(bytes=4 * e * n + 8 * T + 2 * weights, flops=20 * n)
    return dict(bytes=2 * e * n + 8 * T + weights, flops=7 * n)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_delta(case, st):
    """S_t = a_t S_{t-1} + b_t k_t (v_t - a_t S_{t-1}^T k_t)^T,  o_t = scale S_t^T q_t, one token at a
    time; the gradients from the same recurrence run backwards."""
    group = case["Hv"] // case["Hk"]
    q, k = (st[n].double().repeat_interleave(group, -2) for n in ("q", "k"))
    v, al, be, sc = st["v"].double(), st["g"].double().exp(), st["beta"].double(), st["scale"]
    B, L, Hv, Dk, Dv = case["B"], case["L"], case["Hv"], case["Dk"], case["Dv"]
    s = st["s0"].double() if st["s0"] is not None else torch.zeros(B, Hv, Dk, Dv, dtype=torch.float64, device=v.device)
    o = torch.empty(B, L, Hv, Dv, dtype=torch.float64, device=v.device)
    train, seg = case["op"] == "train", 128
    kept = {}

    def advance(s, t):
        s = s * al[:, t, :, None, None]
        e = v[:, t] - torch.einsum("bhkv,bhk->bhv", s, k[:, t])
        return s, e, s + k[:, t, :, :, None] * (be[:, t, :, None] * e)[:, :, None, :]

    for t in range(L):
        if train and t % seg == 0:
            kept[t] = s
        s = advance(s, t)[2]
        o[:, t] = sc * torch.einsum("bhkv,bhk->bhv", s, q[:, t])
    if not train:
        return dict(o=o, s_last=s)
    do = st["do"].double()
    z = st["ds_last"].double() if st["ds_last"] is not None else torch.zeros_like(s)
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, al, be))
    for t0 in sorted(kept, reverse=True):
        x, steps = kept.pop(t0), []
        for t in range(t0, min(L, t0 + seg)):
            faded, e, x = advance(x, t)
            steps.append((t, faded, e, x))
        for t, faded, e, after in reversed(steps):
            dq[:, t] = sc * torch.einsum("bhkv,bhv->bhk", after, do[:, t])
            z = z + sc * q[:, t, :, :, None] * do[:, t, :, None, :]
            u_bar = torch.einsum("bhkv,bhk->bhv", z, k[:, t])
            db[:, t] = (u_bar * e).sum(-1)
            dv[:, t] = be[:, t, :, None] * u_bar
            dk[:, t] = torch.einsum("bhkv,bhv->bhk", z, be[:, t, :, None] * e) - torch.einsum("bhkv,bhv->bhk", faded, dv[:, t])
            z = z - k[:, t, :, :, None] * dv[:, t, :, None, :]
            dg[:, t] = (z * faded).sum((-1, -2))
            z = z * al[:, t, :, None, None]
    share = lambda x: x.reshape(B, L, case["Hk"], group, Dk).sum(3)  # noqa: E731
    out = dict(o=o, s_last=s, dq=share(dq), dk=share(dk), dv=dv, dg=dg, dbeta=db)
    if st["s0"] is not None:
        out["ds0"] = z
    return out


def _exact_turn(case, st, x, back=False):
    """Pairs as complex numbers times amplitude * exp(i position frequency); back: its transpose."""
    n = case["rot"] // 2
    turn = torch.polar(torch.full((), st["amp"], dtype=torch.float64, device=x.device).expand(case["B"], case["L"], n),
                       st["pos"].double()[..., None] * st["freq"])[:, :, None]
    lo, hi = (slice(0, n), slice(n, 2 * n)) if case["layout"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y = torch.complex(x[..., lo], x[..., hi]) * (turn.conj() if back else turn)
    x = x.clone()
    x[..., lo], x[..., hi] = y.real, y.imag
    return x


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "step":
        group = case["Hv"] // case["Hk"]
        q, k = (st[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
        s = st["state"].double() * st["g"].double().exp()[..., None, None]
        e = st["beta"].double()[..., None] * (st["v"].double() - torch.einsum("bhkv,bhk->bhv", s, k))
        s = s + torch.einsum("bhk,bhv->bhkv", k, e)
        return dict(o=st["scale"] * torch.einsum("bhkv,bhk->bhv", s, q), state=s)
    if case["op"] in ("prefill", "train"):
        return _exact_delta(case, st)
    if case["op"] == "rotary":
        return _exact_turn(case, st, st["x"].double())
    out = {}
    for n in ("q", "k"):
        x = st[n].double()
        w = st["w" + n].double() if st["w" + n] is not None else torch.ones(case["D"], dtype=torch.float64, device=x.device)
        count = case["D"] if case["norm"] == "rms" else 1
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / count + st["eps"])
        out[n] = _exact_turn(case, st, x * r * w)
        if case["backward"]:
            dy = _exact_turn(case, st, st["d" + n].double(), back=True)
            dn = dy * w
            out["d" + n] = r * dn - x * r ** 3 * (dn * x).sum(-1, keepdim=True) / count
            if case["norm"] == "rms":
                out["dw" + n] = (dy * x * r).sum((0, 1, 2))
    return out
