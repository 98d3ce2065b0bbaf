"""Plain 64-bit implementations of the sequence operators, token by token,
with a magnitude beside every result: the same formula with every term taken
positive.  A computed value whose factors and sums each lose at most a few
units of 2^-24 is within (number of steps) * 2^-24 of its magnitude, which is
how the tests derive their tolerances."""
import numpy as np

U = 2.0 ** -24
# half a unit in the last place, and half the smallest subnormal step
HALF_ULP = {"f32": (2.0 ** -24, 0.0), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 0.0)}


def sig(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.where(v > 0, v, 0) + np.log1p(np.exp(-np.abs(v)))


def lengths(lens, B, T):
    return [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]


def scan_forward(x, r, i, lam, h0, lens, c):
    """(y, hT, states before each token, magnitude of y, magnitude of hT)."""
    B, T, D = x.shape
    rate = c * softplus(lam)
    y, ym = np.zeros((B, T, D)), np.zeros((B, T, D))
    before = np.zeros((B, T, D))
    hT, hm = np.zeros((B, D)), np.zeros((B, D))
    for b, n in enumerate(lengths(lens, B, T)):
        h = np.zeros(D) if h0 is None else h0[b].copy()
        m = np.abs(h)
        for t in range(n):
            before[b, t] = h
            l = -rate * sig(r[b, t])
            put = np.sqrt(-np.expm1(2 * l)) * sig(i[b, t]) * x[b, t]
            h = np.exp(l) * h + put
            m = np.exp(l) * m + np.abs(put)
            y[b, t], ym[b, t] = h, m
        for t in range(n, T):
            before[b, t] = h
        hT[b], hm[b] = h, m
    return y, hT, before, ym, hm


def scan_backward(dy, dhT, x, r, i, lam, h0, lens, c):
    """({name: gradient}, {name: magnitude})."""
    B, T, D = x.shape
    rate = c * softplus(lam)
    _, _, before, _, _ = scan_forward(x, r, i, lam, h0, lens, c)
    _, _, mbefore, _, _ = scan_forward(np.abs(x), r, i, lam, None if h0 is None else np.abs(h0), lens, c)
    g = {k: np.zeros((B, T, D)) for k in ("dx", "dr", "di")}
    m = {k: np.zeros((B, T, D)) for k in ("dx", "dr", "di")}
    g["dlam"], m["dlam"] = np.zeros(D), np.zeros(D)
    g["dh0"], m["dh0"] = np.zeros((B, D)), np.zeros((B, D))
    for b, n in enumerate(lengths(lens, B, T)):
        gh = np.zeros(D) if dhT is None else dhT[b].copy()
        gm = np.abs(gh)
        for t in reversed(range(n)):
            sr, si = sig(r[b, t]), sig(i[b, t])
            l = -rate * sr
            a, z = np.exp(l), -np.expm1(2 * l)
            s = np.sqrt(z)
            inv = np.divide(1.0, s, out=np.zeros_like(s), where=s > 0)
            gh, gm = gh + dy[b, t], gm + np.abs(dy[b, t])
            ax = np.abs(x[b, t])
            g["dx"][b, t], m["dx"][b, t] = gh * s * si, gm * s * si
            g["di"][b, t] = gh * s * x[b, t] * si * (1 - si)
            m["di"][b, t] = gm * s * ax * si * (1 + si)
            dl = a * gh * before[b, t] - a * a * inv * gh * si * x[b, t]
            dm = a * gm * mbefore[b, t] + a * a * inv * gm * si * ax
            g["dr"][b, t], m["dr"][b, t] = dl * l * (1 - sr), dm * -l * (1 + sr)
            g["dlam"] += dl * -c * sr * sig(lam)
            m["dlam"] += dm * c * sr * sig(lam)
            gh, gm = gh * a, gm * a
        g["dh0"][b], m["dh0"][b] = gh, gm
    return g, m


def conv_forward(x, w, bias, state, lens, act):
    """(y, state_out, pre-activation, magnitude of the pre-activation)."""
    B, T, D = x.shape
    K = w.shape[1]
    ext = np.concatenate([np.zeros((B, K - 1, D)) if state is None else state, x], 1)
    y, u, um, out = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, K - 1, D))
    for b, n in enumerate(lengths(lens, B, T)):
        for t in range(n):
            u[b, t] = (0 if bias is None else bias) + sum(w[:, j] * ext[b, t + j] for j in range(K))
            um[b, t] = (0 if bias is None else np.abs(bias)) + sum(np.abs(w[:, j] * ext[b, t + j]) for j in range(K))
            y[b, t] = u[b, t] * sig(u[b, t]) if act else u[b, t]
        out[b] = ext[b, n:n + K - 1]
    return y, out, u, um


def conv_backward(dy, dstate_out, x, w, bias, state, lens, act):
    B, T, D = x.shape
    K = w.shape[1]
    ext = np.concatenate([np.zeros((B, K - 1, D)) if state is None else state, x], 1)
    _, _, u, um = conv_forward(x, w, bias, state, lens, act)
    de, dem = np.zeros_like(ext), np.zeros_like(ext)
    g = {"dw": np.zeros((D, K)), "dbias": np.zeros(D)}
    m = {"dw": np.zeros((D, K)), "dbias": np.zeros(D)}
    for b, n in enumerate(lengths(lens, B, T)):
        for t in range(n):
            du, dm = dy[b, t].copy(), np.abs(dy[b, t])
            if act:
                s = sig(u[b, t])
                du *= s * (1 + u[b, t] * (1 - s))
                # the factor's own error: sig and u enter it with weights below 1 + |u|
                dm = dm * (1 + um[b, t])
            g["dbias"] += du
            m["dbias"] += dm
            for j in range(K):
                de[b, t + j] += w[:, j] * du
                dem[b, t + j] += np.abs(w[:, j]) * dm
                g["dw"][:, j] += du * ext[b, t + j]
                m["dw"][:, j] += dm * np.abs(ext[b, t + j])
        if dstate_out is not None:
            de[b, n:n + K - 1] += dstate_out[b]
            dem[b, n:n + K - 1] += np.abs(dstate_out[b])
    g["dstate"], m["dstate"] = de[:, :K - 1], dem[:, :K - 1]
    g["dx"], m["dx"] = de[:, K - 1:], dem[:, K - 1:]
    return g, m


def norm_rows(h, w, eps):
    """(v, scale) of the rows of h in 64 bits."""
    ms = (h * h).mean(1, keepdims=True) + eps
    v = np.divide(h, np.sqrt(ms), out=np.zeros_like(h), where=ms > 0) * w
    return v, np.abs(v).max(1) / 127


def check(got, ref, mag, steps, dtype, what):
    """|got - ref| <= half an ulp of the type + steps * 2^-24 * magnitude."""
    got = np.asarray(got, dtype=np.float64)
    rel, absolute = HALF_ULP[dtype]
    lim = rel * np.abs(ref) * 1.01 + absolute + steps * U * mag + 1e-37
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    bad = np.abs(got - ref) > lim
    if bad.any():
        k = int(np.argmax(np.abs(got - ref) - lim))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at flat {k}: got {got.flat[k]!r} "
                             f"ref {ref.flat[k]!r} limit {lim.flat[k]!r}")
