"""The gated scan in 64 bits with an error bound beside every result, followed
channel by channel and token by token.

The bounds, in units of U = 2^-24 (an fp32 rounding):

* a logistic function loses 8 + 2|v|: the approximate exponential (2 units in
  the last place), its argument's two roundings, each |v| in the result, the sum
  and the approximate reciprocal; so does its complement, which is exp(-v) times
  it;
* a log decay l = -rate sig(r) loses 12 + that = 20 + 2|r| of itself, and a decay
  a = exp(l) that times |l| and 4 more;
* sqrt(1 - a^2) loses at most what l does and 12 more; so does its reciprocal;
* a sum or a product of two values loses one unit of its own.

A state's error is then e_t = a e_{t-1} + (loss of a) a |h_{t-1}| + (loss of the
input) |input| + 2 |h_t|, whatever order the tokens are put together in: a fold
of maps rounds no more often than a walk.  The gradients follow in the same way
from the end."""
import numpy as np

import seq_oracle as so

U = so.U


def gates(r, i, lam, c):
    """Per token: dict of the factors and, as *_e, their relative losses."""
    rate = c * so.softplus(lam)
    sr, si = so.sig(r), so.sig(i)
    vr, vi = np.minimum(np.abs(r), 90), np.minimum(np.abs(i), 90)
    l = -rate * sr
    a = np.exp(l)
    s = np.sqrt(-np.expm1(2 * l))
    near = np.where(np.isfinite(l), np.maximum(l, -700), -700)  # past it a is 0, and so is a l
    le = 20 + 2 * vr
    return {"sr": sr, "si": si, "cr": so.sig(-r), "ci": so.sig(-i), "a": a, "al": a * near, "s": s,
            "inv": np.divide(1.0, s, out=np.zeros_like(s), where=s > 0), "rate": rate,
            "l_e": le * U, "a_e": (4 + np.minimum(-near, 200) * le) * U, "s_e": (12 + le) * U, "si_e": (8 + 2 * vi) * U,
            "sr_e": (8 + 2 * vr) * U}


def forward(x, r, i, lam, h0, lens, c):
    """{y, hT, h: (value, bound)}; h is the state before each token, with its
    magnitude as a third."""
    B, T, D = x.shape
    y, ye, hb, hbe, hbm = (np.zeros((B, T, D)) for _ in range(5))
    hT, hTe = np.zeros((B, D)), np.zeros((B, D))
    for b, n in enumerate(so.lengths(lens, B, T)):
        h = np.zeros(D) if h0 is None else h0[b].copy()
        m, e = np.abs(h), np.zeros(D)
        for t in range(n):
            q = gates(r[b, t], i[b, t], lam, c)
            put = q["s"] * q["si"] * x[b, t]
            hb[b, t], hbe[b, t], hbm[b, t] = h, e, m
            e = q["a"] * e + q["a_e"] * q["a"] * m + (q["s_e"] + q["si_e"] + 3 * U) * np.abs(put) + 1e-18 * np.abs(x[b, t])
            h, m = q["a"] * h + put, q["a"] * m + np.abs(put)
            e = e + 2 * U * m
            y[b, t], ye[b, t] = h, e
        hT[b], hTe[b] = h, e
    return {"y": (y, ye), "hT": (hT, hTe), "h": (hb, hbe, hbm)}


def backward(dy, dhT, x, r, i, lam, h0, lens, c):
    """{dx, dr, di, dlam, dh0: (value, bound)}."""
    B, T, D = x.shape
    h, he, hm = forward(x, r, i, lam, h0, lens, c)["h"]
    o = {k: (np.zeros((B, T, D)), np.zeros((B, T, D))) for k in ("dx", "dr", "di")}
    dlam, dlame, dlamm, terms = np.zeros(D), np.zeros(D), np.zeros(D), 0
    dh0, dh0e = np.zeros((B, D)), np.zeros((B, D))
    for b, n in enumerate(so.lengths(lens, B, T)):
        g = np.zeros(D) if dhT is None else dhT[b].copy()
        gm, ge = np.abs(g), np.zeros(D)
        for t in reversed(range(n)):
            q = gates(r[b, t], i[b, t], lam, c)
            g, gm = g + dy[b, t], gm + np.abs(dy[b, t])
            ge = ge + 2 * U * gm
            ax = np.abs(x[b, t])
            f = q["s"] * q["si"]
            o["dx"][0][b, t], o["dx"][1][b, t] = g * f, f * (ge + (q["s_e"] + q["si_e"] + 3 * U) * gm)
            k = f * ax * q["ci"]
            o["di"][0][b, t] = g * f * x[b, t] * q["ci"]
            o["di"][1][b, t] = k * (ge + (q["s_e"] + 2 * q["si_e"] + 5 * U) * gm)
            # dl / a = g (h - a / s sig(i) x); the second term and its factors' losses
            put = q["a"] * q["inv"] * q["si"]
            v, vm = h[b, t] - put * x[b, t], hm[b, t] + put * ax
            ve = he[b, t] + put * ax * (q["a_e"] + q["s_e"] + q["si_e"] + q["sr_e"] + 5 * U) + (q["sr_e"] + 3 * U) * hm[b, t]
            we = ge * vm + gm * ve + (q["a_e"] + 2 * U) * gm * vm  # of g v, with the loss of a before it
            o["dr"][0][b, t] = g * v * q["al"] * q["cr"]
            o["dr"][1][b, t] = np.abs(q["al"]) * q["cr"] * (we + (q["l_e"] + q["sr_e"] + 5 * U) * gm * vm)
            w = c * q["sr"] * q["a"] * so.sig(lam)
            dlam -= g * v * w
            dlamm += gm * vm * w
            dlame += w * (we + (q["sr_e"] + 12 * U) * gm * vm)
            terms += 1
            ge = q["a"] * ge + (q["a_e"] + U) * q["a"] * gm
            g, gm = g * q["a"], gm * q["a"]
        dh0[b], dh0e[b] = g, ge + U * gm
    return {**o, "dlam": (dlam, dlame + terms * U * dlamm), "dh0": (dh0, dh0e)}


def check(got, ref, bound, dtype, what):
    """|got - ref| <= half an ulp of the type + the bound (and fp32's smallest values)."""
    got = np.asarray(got, dtype=np.float64)
    rel, absolute = so.HALF_ULP[dtype]
    lim = rel * (np.abs(ref) + bound) + absolute + bound + 1e-37
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    bad = np.abs(got - ref) > lim
    if bad.any():
        k = int(np.argmax(np.abs(got - ref) / lim))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; at flat {k}: got {got.flat[k]!r} "
                             f"ref {ref.flat[k]!r} limit {lim.flat[k]!r}")
