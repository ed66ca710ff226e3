"""Plain float64 forms of the gated delta rule and of the rotation with norms,
one token at a time, for the tests of the CUDA calls (numpy, no framework code)."""
import numpy as np


def _group(x, Hv):
    return np.repeat(x, Hv // x.shape[-2], axis=-2)


def decay(g):
    with np.errstate(over="ignore"):
        return np.exp(np.asarray(g, np.float64))


def delta_forward(q, k, v, g, beta, s0, scale):
    """o, s_last, and per token (faded state, e, state after)."""
    B, L, Hv, Dv = v.shape
    q, k = _group(q, Hv), _group(k, Hv)
    s = np.zeros((B, Hv, q.shape[-1], Dv)) if s0 is None else np.asarray(s0, np.float64)
    a = decay(g)
    o, steps = np.zeros(v.shape), []
    for t in range(L):
        faded = a[:, t, :, None, None] * s
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", faded, k[:, t])
        s = faded + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None, :]
        o[:, t] = scale * np.einsum("bhkv,bhk->bhv", s, q[:, t])
        steps.append((faded, e, s))
    return o, s, steps


def delta_backward(q, k, v, g, beta, s0, scale, do, ds_last):
    B, L, Hv, Dv = v.shape
    Hk, Dk = q.shape[-2:]
    _, _, steps = delta_forward(q, k, v, g, beta, s0, scale)
    qg, kg, a = _group(q, Hv), _group(k, Hv), decay(g)
    z = np.zeros((B, Hv, Dk, Dv)) if ds_last is None else np.array(ds_last, np.float64)
    dq, dk = np.zeros(qg.shape), np.zeros(kg.shape)
    dv, dg, db = np.zeros(v.shape), np.zeros(g.shape), np.zeros(g.shape)
    for t in reversed(range(L)):
        faded, e, after = steps[t]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", after, do[:, t])
        z = z + scale * qg[:, t, :, :, None] * do[:, t, :, None, :]
        x = np.einsum("bhkv,bhk->bhv", z, kg[:, t])
        db[:, t] = (x * e).sum(-1)
        dv[:, t] = beta[:, t, :, None] * x
        dk[:, t] = np.einsum("bhkv,bhv->bhk", z, beta[:, t, :, None] * e) - np.einsum("bhkv,bhv->bhk", faded, dv[:, t])
        z = z - kg[:, t, :, :, None] * dv[:, t, :, None, :]
        dg[:, t] = (z * faded).sum((-1, -2))
        z = a[:, t, :, None, None] * z
    share = lambda x: x.reshape(B, L, Hk, Hv // Hk, Dk).sum(3)  # noqa: E731
    return dict(dq=share(dq), dk=share(dk), dv=dv, dg=dg, dbeta=db, ds0=z)


def turn(x, pos, freq, layout, amp, back=False):
    """Rotated pairs as complex numbers; back: the transpose."""
    n = len(freq)
    ang = np.asarray(pos, np.float64)[..., None] * freq
    w = amp * np.exp(1j * (-ang if back else ang))[..., None, :]
    lo, hi = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    c = (x[..., lo] + 1j * x[..., hi]) * w
    y = np.array(x, np.float64)
    y[..., lo], y[..., hi] = c.real, c.imag
    return y


def norm(x, w, kind, eps):
    if kind is None:
        r, count = np.ones(x.shape[:-1] + (1,)), None
    else:
        count = x.shape[-1] if kind == "rms" else 1
        with np.errstate(divide="ignore"):
            r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / count + eps)
    return x * r * (1.0 if w is None else w), r, count


def norm_turn_backward(x, w, kind, eps, pos, freq, layout, amp, dy):
    dz = turn(dy, pos, freq, layout, amp, back=True)
    _, r, count = norm(x, None, kind, eps)
    dn = dz * (1.0 if w is None else w)
    dx = r * dn
    if count is not None:
        dx = dx - x * r ** 3 * (dn * x).sum(-1, keepdims=True) / count
    return dx, (dz * x * r).reshape(-1, x.shape[-1]).sum(0)
