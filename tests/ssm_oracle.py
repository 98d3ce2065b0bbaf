"""The selective scan in 64 bits, token by token, with an error bound beside every
result, and its gradients from the adjoint.

The bounds, in units of U = 2^-24 (an fp32 rounding, relative to the value):

* the approximate exponential loses 4 (2^-22), and what its argument lost times the
  argument; a reciprocal 2;
* a step softplus(v) loses 16 + 3|v|: exp(-|v|) (4, and |v| for each of three roundings of
  its argument), the quotient and the series (12); without softplus 1;
* a decay a = exp(s A) loses 5 + |s A| (3 + the step's loss);
* a logistic function loses 8 + 2|z|;
* a sum of n values loses n of the sum of their magnitudes, in whatever order.

A state's error is then e_t = a e_{t-1} + (loss of a) a |h_{t-1}| + (loss of the input) |input| + |h_t|.
Where the walk over time is split, a part's decay is exp(A sum s) with a sum of as many
roundings as tokens: at most |l| exp(-|l|) <= 0.37 of that many, of the largest state, come on top."""
import numpy as np

U = 2.0 ** -24
EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
TINY = {"f32": 2.0 ** -140, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}  # half a step below the normal numbers


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def sig(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def scan(x, delta, A, Bm, Cm, skip=None, z=None, bias=None, h0=None, lens=None, dy=None, dhT=None, groups=1, soft=True, parts=True):
    """dicts (value, bound) of y, hT and, with dy, of the gradients; the bounds without the last
    rounding to the outputs' type.  parts: the walk may be split."""
    B, T, D = x.shape
    N, per = A.shape[1], D // groups
    lens = [T] * B if lens is None else [min(max(int(n), 0), T) for n in lens]
    live = np.zeros((B, T, 1))
    for b, n in enumerate(lens):
        live[b, :n] = 1
    clean = [np.where(live > 0, t, 0.0) if t is not None else None for t in (x, delta, Bm, Cm, z, dy)]  # NaN past the ends
    x, delta, Bm, Cm, z, dy = clean
    skip = np.zeros(D) if skip is None else skip
    v = delta + (0 if bias is None else bias)
    s = (softplus(v) if soft else v) * live
    es = 16 + 3 * np.minimum(np.abs(v), 90) if soft else np.ones_like(v)
    Bc = np.repeat(Bm.reshape(B, T, groups, N), per, 2)
    Cc = np.repeat(Cm.reshape(B, T, groups, N), per, 2)
    l = s[..., None] * A
    a, ea = np.exp(l), 5 + np.abs(l) * (3 + es[..., None])
    u = s * x
    put = u[..., None] * Bc
    h, e = (np.zeros((B, D, N)) if h0 is None else h0), np.zeros((B, D, N))
    first = h
    hs, he = [], []
    for t in range(T):
        on = live[:, t, :, None]
        new = a[:, t] * h + put[:, t]
        ne = a[:, t] * e + ea[:, t] * np.abs(a[:, t] * h) + (es[:, t, :, None] + 3) * np.abs(put[:, t]) + np.abs(new)
        h, e = np.where(on > 0, new, h), np.where(on > 0, ne, e)
        hs.append(h)
        he.append(e)
    hs, he = np.stack(hs, 1), np.stack(he, 1)
    big = np.maximum(np.abs(hs).max(1, keepdims=True), np.abs(first)[:, None])
    fold = 0.4 * T if parts else 0.0
    he = he + fold * big
    o = (hs * Cc).sum(-1) + skip * x
    oe = (np.abs(Cc) * he + (N + 2) * np.abs(hs * Cc)).sum(-1) + 2 * np.abs(skip * x)
    if z is None:
        gate, ge = np.ones_like(x), 0.0
    else:
        gate, ge = z * sig(z), 8 + 2 * np.minimum(np.abs(z), 90)
    out = {"y": (o * gate * live, (oe * np.abs(gate) + (ge + 3) * np.abs(o * gate)) * live), "hT": (hs[:, -1], he[:, -1])}
    if dy is None:
        return out
    go, goe = dy * gate, (ge + 2) * np.abs(dy * gate)
    g, e = (np.zeros((B, D, N)) if dhT is None else dhT), np.zeros((B, D, N))
    before = np.concatenate([first[:, None], hs[:, :-1]], 1)
    be = np.concatenate([np.zeros_like(he[:, :1]), he[:, :-1]], 1)
    gs, gse, qs, qse = (np.zeros((B, T, D, N)) for _ in range(4))
    most = np.abs(g)
    ags, agse = [None] * T, [None] * T
    for t in reversed(range(T)):
        on = live[:, t, :, None] > 0
        gt = Cc[:, t] * go[:, t, :, None] + g
        gte = np.abs(Cc[:, t]) * goe[:, t, :, None] + e + 2 * np.abs(gt)
        ag = a[:, t] * gt
        age = a[:, t] * gte + (ea[:, t] + 1) * np.abs(ag)
        gs[:, t], gse[:, t] = np.where(on, gt, 0), np.where(on, gte, 0)
        ags[t], agse[t] = np.where(on, ag, 0), np.where(on, age, 0)
        g, e = np.where(on, ag, g), np.where(on, age, e)
        most = np.maximum(most, np.abs(gt))
    extra = fold * most[:, None]
    gse = gse + extra * live[..., None]
    ags, agse = np.stack(ags, 1), np.stack(agse, 1) + extra * live[..., None] * a
    qs = ags * before
    qse = agse * np.abs(before) + np.abs(ags) * be + np.abs(qs)
    depth = 32 + D // 8  # lanes, warps and blocks that a sum over channels goes through, with room

    def mix(v):
        return v.reshape(B, T, groups, per, N).sum(3).reshape(B, T, groups * N)

    w = gs * u[..., None]
    out["dBm"] = mix(w), mix(gse * np.abs(u[..., None]) + (es[..., None] + 2 + depth) * np.abs(w))
    w = hs * go[..., None]
    out["dCm"] = mix(w) * live, mix(he * np.abs(go[..., None]) + np.abs(hs) * goe[..., None] + depth * np.abs(w)) * live
    du, due = (gs * Bc).sum(-1), (gse * np.abs(Bc) + (N + 2) * np.abs(gs * Bc)).sum(-1)
    ds, dse = (qs * A).sum(-1), (qse * np.abs(A) + (N + 5) * np.abs(qs * A)).sum(-1)
    out["dx"] = (du * s + go * skip) * live, (due * s + du.__abs__() * s * (es + 2) + (goe + 2 * np.abs(go)) * np.abs(skip)) * live
    f = sig(v) if soft else np.ones_like(v)
    fe = 8 + 3 * np.minimum(np.abs(v), 90) if soft else 0.0
    dv = (ds + du * x) * f * live
    dve = ((dse + due * np.abs(x) + 3 * (np.abs(ds) + np.abs(du * x))) * f + fe * np.abs(dv)) * live
    out["ddelta"] = dv, dve
    tokens = B * T + 64
    out["dbias"] = dv.sum((0, 1)), (dve + tokens * np.abs(dv)).sum((0, 1))
    out["dskip"] = (go * x).sum((0, 1)), ((goe + tokens * np.abs(go)) * np.abs(x)).sum((0, 1))
    w = qs * s[..., None]
    out["dA"] = w.sum((0, 1)), (qse * s[..., None] + (es[..., None] + 2 + tokens) * np.abs(w)).sum((0, 1))
    out["dh0"] = g, e + fold * most
    if z is not None:
        f = sig(z) * (1 + z * (1 - sig(z)))
        fe = sig(z) * (1 + np.abs(z)) * (ge + 6)
        out["dz"] = dy * o * f * live, (np.abs(dy) * (oe * np.abs(f) + np.abs(o) * (fe + 3 * np.abs(f)))) * live
    return out


def close(got, ref, dtype, what):
    """got within the bound of ref, plus the rounding to dtype."""
    value, bound = ref
    assert got.shape == value.shape, (what, got.shape, value.shape)
    lim = bound * U * 1.01 + np.abs(value) * EPS[dtype] * 1.01 + TINY[dtype] + 1e-36
    bad = ~(np.abs(got - value) <= lim)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(got - value) / lim, 0)), bad.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {at} got {got[at]!r} ref {value[at]!r} lim {lim[at]:.3g}")
