"""The scan's error bounds (seq_bounds.py): their values are the oracle's, an
fp32 walk of the formulas stays inside them, and the mistakes that they are there
to find do not."""
import numpy as np
import pytest

import seq_bounds as sb
import seq_oracle as so

C = 8.0
f = np.float32


def case(T, D=8, seed=0, lo=-1.0, hi=1.0, slow=True):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s).astype(f).astype(float)  # noqa: E731
    u = g.uniform(0.9, 0.999, D) if slow else g.uniform(0.02, 0.999, D)
    return {"x": n(1, T, D), "r": g.uniform(lo, hi, (1, T, D)).astype(f).astype(float),
            "i": g.uniform(lo, hi, (1, T, D)).astype(f).astype(float), "dy": n(1, T, D), "dhT": n(1, D), "h0": n(1, D),
            "lam": np.log(np.expm1(-np.log(u) / C)).astype(f).astype(float)}


def walk(s, round_state=lambda h: h, complement=lambda v, sig: np.exp(-v) * sig):
    """The formulas in fp32, one sequence; (y, hT, di, dr)."""
    x, r, i, dy = (s[k][0].astype(f) for k in ("x", "r", "i", "dy"))
    lam, T = s["lam"].astype(f), s["x"].shape[1]
    sig = lambda v: f(1) / (f(1) + np.exp(-v))  # noqa: E731
    rate = f(C) * np.log1p(np.exp(lam))
    sr, si = sig(r), sig(i)
    l = -rate * sr
    a, q = np.exp(l), np.sqrt(-np.expm1(f(2) * l))
    h, hs = s["h0"][0].astype(f), []
    for t in range(T):
        hs.append(h)
        h = round_state(a[t] * h + q[t] * si[t] * x[t]).astype(f)
    y, g = np.stack(hs[1:] + [h]), s["dhT"][0].astype(f)
    di, dr = np.zeros_like(x), np.zeros_like(x)
    for t in reversed(range(T)):
        g = g + dy[t]
        di[t] = g * q[t] * si[t] * x[t] * complement(i[t], si[t])
        dl = a[t] * g * hs[t] - a[t] * a[t] / q[t] * g * si[t] * x[t]
        dr[t] = dl * l[t] * complement(r[t], sr[t])
        g = g * a[t]
    return y, h, di, dr


def inside(s, got):
    want = {**sb.forward(s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C),
            **sb.backward(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C)}
    for k, v in zip(("y", "hT", "di", "dr"), got):
        sb.check(v[None], *want[k], "f32", k)


def test_values_are_the_oracles():
    s = case(60, slow=False)
    y, hT, _, _, _ = so.scan_forward(s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C)
    g, _ = so.scan_backward(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C)
    mine = {**sb.forward(s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C),
            **sb.backward(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C)}
    for k, v in {"y": y, "hT": hT, **g}.items():
        assert np.allclose(mine[k][0], v, rtol=1e-11, atol=1e-14), k


@pytest.mark.parametrize("slow", [True, False])
@pytest.mark.parametrize("lo,hi", [(-1, 1), (6, 28), (-28, -6)])
def test_an_fp32_walk_is_inside(slow, lo, hi):
    s = case(300, lo=lo, hi=hi, slow=slow)
    inside(s, walk(s))


def test_a_16_bit_state_is_outside():
    s = case(4000)
    inside(s, walk(s))
    with pytest.raises(AssertionError, match="y|hT"):
        inside(s, walk(s, round_state=lambda h: h.astype(np.float16)))


def test_a_complement_by_subtraction_is_outside():
    s = case(60, lo=8, hi=28)
    with pytest.raises(AssertionError, match="di"):
        inside(s, walk(s, complement=lambda v, sig: f(1) - sig))


def test_an_infinite_rate_has_its_limit():
    s = case(20)
    s["lam"][3] = np.inf
    q = {**sb.forward(s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C),
         **sb.backward(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], s["h0"], None, C)}
    assert all(np.isfinite(v).all() and np.isfinite(e).all() for v, e, *_ in q.values())
    assert np.array_equal(q["y"][0][0, :, 3], (so.sig(s["i"]) * s["x"])[0, :, 3]) and not q["dr"][0][..., 3].any()
