"""Plain float64 forms of the gated recurrence, the short convolution and layer norm of a sum, token by token (numpy, no
framework code), each output with a bound on what 32-bit arithmetic in any order of its sums may be off by.

U = 2^-24 is a rounding of a 32-bit value.  The machine's own functions: exp2 2^-22 = 4 U, 1/x 2^-23 = 2 U, 1/sqrt(x)
2^-22.4 < 4 U.  A sigmoid of g then is off by (|g| + 8) U relative: the product in front of exp2 (|g| U), exp2, 1 + e,
1/x.  Sums are bounded by the sums of their terms' sizes, so that the bounds hold for every association."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}       # half a step of the output's type, relative


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def _gates(x, ga, gx, rate, reset, valid, normalize):
    """Per value a, n, s, u and the relative errors of a, n u and a^2 u / n."""
    r = sigmoid(ga)
    la = -rate * r
    a, m = np.exp(la), -np.expm1(la)
    n = np.sqrt(-np.expm1(2 * la)) if normalize else np.ones_like(a)
    s = np.ones_like(x) if gx is None else sigmoid(gx)
    ds = np.zeros_like(x) if gx is None else (np.abs(gx) + 8) * U
    dr = (np.abs(ga) + 8) * U
    far = la < -0.24
    # a = 1 - m, m = 1 - exp(la): near one a rounding; further off exp2's 4 U of a and the two subtractions' U of 1 and of
    # m, absolute, so 2 U / a relative
    da = np.abs(la) * (dr + 5 * U) + np.where(far, 5 + 2 / np.maximum(a, 1e-30), 1) * U
    dm = np.where(far, a / np.maximum(m, 0.2) * da + U, dr + 5 * U)
    dn = dm + 7 * U if normalize else 0 * dm
    with np.errstate(divide="ignore", invalid="ignore"):
        slope = np.where(n > 0, a * a / n, 0.0) if normalize else np.zeros_like(a)
    if reset is not None:
        a, n = np.where(reset[..., None], 0.0, a), np.where(reset[..., None], 1.0, n)
        slope = np.where(reset[..., None], 0.0, slope)
    if valid is not None:
        a, n = np.where(valid[..., None], a, 1.0), np.where(valid[..., None], n, 0.0)
        slope = np.where(valid[..., None], slope, 0.0)
        da = np.where(valid[..., None], da, 0.0)
    return r, dr, a, da, n, s, ds, s * x, dn + ds + 3 * U, slope, 2 * da + dn + ds + 8 * U


def _valid(lengths, B, L):
    return None if lengths is None else np.arange(L) < np.clip(lengths, 0, L)[:, None]


def scan(x, ga, gx, rate, h0=None, reset=None, lengths=None, normalize=True, dh=None, dh_last=None, depth=160):
    """Values and bounds: {"h": (value, bound), ...}; with dh the gradients too.  depth: roundings of drate's sum."""
    B, L, C = x.shape
    valid = _valid(lengths, B, L)
    clean = (lambda t: t) if valid is None else (lambda t: np.where(valid[..., None], t, 0.0))
    x, ga = clean(x), clean(ga)
    gx = None if gx is None else clean(gx)
    r, dr, a, da, n, s, ds, u, de, slope, dslope = _gates(x, ga, gx, rate, reset, valid, normalize)
    e = n * u
    h = np.zeros((B, C)) if h0 is None else np.array(h0, np.float64)
    size, off = np.abs(h), np.zeros((B, C))
    hs, before, before_size, before_off, offs = (np.zeros((B, L, C)) for _ in range(5))
    for t in range(L):
        fresh = np.zeros((B, 1), bool) if reset is None else (reset[:, t] if valid is None else reset[:, t] & valid[:, t])[:, None]
        h, size, off = (np.where(fresh, 0.0, v) for v in (h, size, off))
        before[:, t], before_size[:, t], before_off[:, t] = h, size, off
        off = a[:, t] * off + a[:, t] * size * (da[:, t] + 2 * U) + np.abs(e[:, t]) * (de[:, t] + 2 * U)
        h, size = a[:, t] * h + e[:, t], a[:, t] * size + np.abs(e[:, t])
        off = off + 2 * U * size
        hs[:, t], offs[:, t] = h, off
    out = dict(h=(clean(hs), clean(offs)), h_last=(h, off + U * np.abs(h)))
    if dh is None:
        return out
    dh = clean(dh)
    z = np.zeros((B, C)) if dh_last is None else np.array(dh_last, np.float64)
    zsize, zoff = np.abs(z), np.zeros((B, C))
    G, Goff = np.zeros((B, L, C)), np.zeros((B, L, C))
    for t in reversed(range(L)):
        fresh = np.zeros((B, 1), bool) if reset is None else (reset[:, t] if valid is None else reset[:, t] & valid[:, t])[:, None]
        G[:, t], gsize = z + dh[:, t], zsize + np.abs(dh[:, t])
        Goff[:, t] = zoff + 2 * U * gsize
        zoff = np.where(fresh, 0.0, a[:, t] * Goff[:, t] + a[:, t] * gsize * (da[:, t] + 2 * U))
        z, zsize = np.where(fresh, 0.0, a[:, t] * G[:, t]), np.where(fresh, 0.0, a[:, t] * gsize)
    past, root = a * before, slope * u
    D = past - root
    doff = a * before_off + a * before_size * (da + 2 * U) + np.abs(root) * dslope + U * (np.abs(past) + np.abs(root))
    dead = np.zeros((B, L), bool) if reset is None else np.array(reset, bool)
    if valid is not None:
        dead = dead | ~valid
    D, doff = np.where(dead[..., None], 0.0, D), np.where(dead[..., None], 0.0, doff)
    dla = G * D
    loff = np.abs(G) * doff + Goff * np.abs(D) + Goff * doff + U * np.abs(dla)
    t, toff = dla * r, loff * r + np.abs(dla) * r * (dr + U)
    out["drate"] = (-t.sum((0, 1)), toff.sum((0, 1)) + depth * U * np.abs(t).sum((0, 1)))
    out["dgate_a"] = (-rate * t * (1 - r), rate * (toff * (1 - r) + (np.abs(t) + toff) * (r * dr + U)) + 4 * U * np.abs(rate * t))
    dx = G * n * s
    xoff = Goff * n * s + np.abs(dx) * (de + 3 * U) + Goff * n * s * de
    out["dx"] = (clean(dx), clean(xoff))
    if gx is not None:
        out["dgate_x"] = (clean(dx * x * (1 - s)), clean(np.abs(x) * (xoff * (1 - s) + (np.abs(dx) + xoff) * (s * ds + U)) + 4 * U * np.abs(dx * x)))
    if h0 is not None:
        out["dh0"] = (z, zoff + U * np.abs(z))
    return out


def _seen(reset, B, L, K):
    """[B, L, K] whether tap j of a token meets its own sequence, and [B, K-1] which inputs go on to the next call."""
    age = np.full((B, L), K)
    for b in range(B):
        a = K
        for t in range(L):
            a = 0 if reset is not None and reset[b, t] else min(a + 1, K)
            age[b, t] = a
    return age, age[..., None] >= np.arange(K - 1, -1, -1)


def conv(x, w, bias=None, silu=False, past=None, reset=None, lengths=None, dy=None, dpast_out=None, depth=300):
    B, L, C = x.shape
    K = w.shape[1]
    valid = _valid(lengths, B, L)
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    clean = (lambda t: t) if valid is None else (lambda t: np.where(valid[..., None], t, 0.0))
    x = clean(x)
    reset = None if reset is None else (reset if valid is None else reset & valid)
    line = np.concatenate([np.zeros((B, K - 1, C)) if past is None else past, x], 1)
    age, seen = _seen(reset, B, L, K)
    win = np.stack([np.where(seen[:, :, j, None], line[:, j:j + L], 0.0) for j in range(K)], 2)   # [B,L,K,C]
    b = np.zeros(C) if bias is None else bias
    p = np.einsum("blkc,ck->blc", win, w) + b
    poff = (K + 1) * U * (np.einsum("blkc,ck->blc", np.abs(win), np.abs(w)) + np.abs(b))
    g = sigmoid(p) if silu else np.ones_like(p)
    dg = (np.abs(p) + 8) * U if silu else 0 * p
    y = p * g
    out = dict(y=(clean(y), clean(1.1 * poff + np.abs(y) * (dg + 2 * U))))
    last, keep = np.zeros((B, K - 1, C)), np.zeros((B, K - 1), bool)
    for i in range(B):
        for j in range(K - 1):
            t = n[i] - (K - 1) + j
            cut = reset is not None and reset[i, max(t + 1, 0):n[i]].any()
            keep[i, j] = not cut
            if not cut:
                last[i, j] = line[i, t + K - 1]
    out["past_out"] = (last, 0 * last)
    if dy is None:
        return out
    dy = clean(dy)
    dp = dy * (g * (1 + p * (1 - g)) if silu else 1.0)
    # act' moves by at most 0.5 with p; its own terms 1 and p (1 - g) by the sigmoid's error and 3 roundings
    dpoff = np.abs(dy) * (0.5 * poff + (1 + np.abs(p)) * (dg + 3 * U)) if silu else 0 * dy
    dline, loff, lsize = (np.zeros_like(line) for _ in range(3))
    dw, woff = np.zeros((C, K)), np.zeros((C, K))
    for j in range(K):
        d, o = np.where(seen[:, :, j, None], dp, 0.0), np.where(seen[:, :, j, None], dpoff, 0.0)
        dline[:, j:j + L] += d * w[:, j]
        loff[:, j:j + L] += o * np.abs(w[:, j])
        lsize[:, j:j + L] += np.abs(d * w[:, j])
        dw[:, j] = (d * line[:, j:j + L]).sum((0, 1))
        woff[:, j] = (o * np.abs(line[:, j:j + L])).sum((0, 1)) + depth * U * np.abs(d * line[:, j:j + L]).sum((0, 1))
    if dpast_out is not None:
        for i in range(B):
            for j in range(K - 1):
                if keep[i, j]:
                    dline[i, n[i] + j] += dpast_out[i, j]
                    lsize[i, n[i] + j] += np.abs(dpast_out[i, j])
    loff += (K + 2) * U * lsize
    out.update(dx=(dline[:, K - 1:], loff[:, K - 1:]), dweight=(dw, woff))
    if bias is not None:
        out["dbias"] = (dp.sum((0, 1)), dpoff.sum((0, 1)) + depth * U * np.abs(dp).sum((0, 1)))
    if past is not None:
        out["dpast"] = (dline[:, :K - 1], loff[:, :K - 1])
    return out


def norm(x, weight=None, bias=None, residual=None, eps=1e-5, depth=80):
    """y, total, mean, inv with bounds; depth: roundings of a row's sum."""
    H = x.shape[-1]
    s = x if residual is None else x + residual
    soff = 0 * s if residual is None else U * np.abs(s)
    mean = s.mean(-1, keepdims=True)
    moff = depth * U * np.abs(s).mean(-1, keepdims=True) + soff.mean(-1, keepdims=True)
    c = s - mean
    coff = soff + moff + U * (np.abs(c) + moff)
    var = (c * c).mean(-1, keepdims=True)
    voff = 2 * (np.abs(c) * coff).mean(-1, keepdims=True) + (coff * coff).mean(-1, keepdims=True) + depth * U * var
    inv = 1 / np.sqrt(var + eps)
    ioff = inv * (0.5 * voff / (var + eps) + 4 * U)
    n = c * inv
    noff = inv * coff + np.abs(c) * ioff + coff * ioff + U * np.abs(n)
    w = np.ones(H) if weight is None else weight
    b = np.zeros(H) if bias is None else bias
    y = n * w + b
    return dict(y=(y, np.abs(w) * noff + 2 * U * (np.abs(n * w) + np.abs(b))), total=(s, soff), mean=(mean[..., 0], moff[..., 0]),
                inv=(inv[..., 0], ioff[..., 0]))


def norm_backward(total, dy, mean, inv, weight=None, dtotal=None, depth=80, rows_depth=400):
    """Gradients of the norm of `total` (the sum, not rounded) with the given mean and inv [N]."""
    H = total.shape[-1]
    w = np.ones(H) if weight is None else weight
    m, i = mean[..., None], inv[..., None]
    n = (total - m) * i
    noff = 3 * U * np.abs(n) + U * np.abs(total) * i     # the difference, the product and one to spare; the sum's rounding
    g = dy * w
    s1, s2 = g.mean(-1, keepdims=True), (g * n).mean(-1, keepdims=True)
    o1 = depth * U * np.abs(g).mean(-1, keepdims=True)
    o2 = depth * U * np.abs(g * n).mean(-1, keepdims=True) + (np.abs(g) * noff).mean(-1, keepdims=True)
    dx = i * (g - s1 - n * s2)
    off = i * (U * np.abs(g) + o1 + np.abs(n) * o2 + noff * np.abs(s2) + 4 * U * (np.abs(g) + np.abs(s1) + np.abs(n * s2)))
    if dtotal is not None:
        dx = dx + dtotal
        off = off + U * (np.abs(dx) + np.abs(dtotal))
    flat = lambda t: t.reshape(-1, H)  # noqa: E731
    dw, db = flat(dy * n), flat(dy)
    return dict(dx=(dx, off), dweight=(dw.sum(0), flat(np.abs(dy) * noff).sum(0) + rows_depth * U * np.abs(dw).sum(0)),
                dbias=(db.sum(0), rows_depth * U * np.abs(db).sum(0)))


def differences(loss, x, step=1e-6):
    """Central differences of loss(**x) by every value of every array of x."""
    out = {}
    for name in x:
        d = np.zeros(x[name].shape)
        for i in np.ndindex(*d.shape):
            v = []
            for sign in (step, -step):
                moved = dict(x, **{name: x[name].copy()})
                moved[name][i] += sign
                v.append(loss(**moved))
            d[i] = (v[0] - v[1]) / (2 * step)
        out[name] = d
    return out
