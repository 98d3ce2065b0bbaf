"""The 64-bit oracle of the sequence operators: gradients against central
differences, and the properties that fix the forward formulas."""
import numpy as np
import pytest

import seq_oracle as so


def _scan(seed, B=2, T=7, D=3):
    g = np.random.default_rng(seed)
    v = {"x": g.normal(size=(B, T, D)), "r": g.normal(size=(B, T, D)), "i": g.normal(size=(B, T, D)),
         "lam": g.normal(size=D) - 2, "h0": g.normal(size=(B, D))}
    return v, g.normal(size=(B, T, D)), g.normal(size=(B, D))


@pytest.mark.parametrize("lens", [None, [7, 0], [4, 1]])
def test_scan_gradients_against_differences(lens):
    v, dy, dhT = _scan(1)

    def loss(**kw):
        w = {**v, **kw}
        y, hT, *_ = so.scan_forward(w["x"], w["r"], w["i"], w["lam"], w["h0"], lens, 8.0)
        return (y * dy).sum() + (hT * dhT).sum()

    g, _ = so.scan_backward(dy, dhT, v["x"], v["r"], v["i"], v["lam"], v["h0"], lens, 8.0)
    eps = 1e-6
    for name, key in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("h0", "dh0")):
        for k in range(v[name].size):
            up, dn = v[name].copy(), v[name].copy()
            up.flat[k] += eps
            dn.flat[k] -= eps
            diff = (loss(**{name: up}) - loss(**{name: dn})) / (2 * eps)
            # truncation eps^2 * third derivative, rounding 2^-52 / eps
            assert abs(diff - g[key].flat[k]) < 1e-7, (name, k)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("lens", [None, [5, 0], [2, 1]])
@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_gradients_against_differences(act, lens, K):
    r = np.random.default_rng(2)
    B, T, D = 2, 5, 3
    v = {"x": r.normal(size=(B, T, D)), "w": r.normal(size=(D, K)), "bias": r.normal(size=D),
         "state": r.normal(size=(B, K - 1, D))}
    dy, ds = r.normal(size=(B, T, D)), r.normal(size=(B, K - 1, D))

    def loss(**kw):
        w = {**v, **kw}
        y, out, _, _ = so.conv_forward(w["x"], w["w"], w["bias"], w["state"], lens, act)
        return (y * dy).sum() + (out * ds).sum()

    g, _ = so.conv_backward(dy, ds, v["x"], v["w"], v["bias"], v["state"], lens, act)
    eps = 1e-6
    for name, key in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("state", "dstate")):
        for k in range(v[name].size):
            up, dn = v[name].copy(), v[name].copy()
            up.flat[k] += eps
            dn.flat[k] -= eps
            diff = (loss(**{name: up}) - loss(**{name: dn})) / (2 * eps)
            assert abs(diff - g[key].flat[k]) < 1e-7, (name, k)


def test_scan_in_two_parts_is_the_whole():
    v, _, _ = _scan(3, T=9)
    y, hT, *_ = so.scan_forward(v["x"], v["r"], v["i"], v["lam"], v["h0"], None, 8.0)
    a = [v[k][:, :4] for k in ("x", "r", "i")]
    b = [v[k][:, 4:] for k in ("x", "r", "i")]
    y1, h1, *_ = so.scan_forward(*a, v["lam"], v["h0"], None, 8.0)
    y2, h2, *_ = so.scan_forward(*b, v["lam"], h1, None, 8.0)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.allclose(h2, hT, atol=1e-14)


def test_conv_state_continues_the_sequence():
    r = np.random.default_rng(4)
    x, w = r.normal(size=(2, 8, 3)), r.normal(size=(3, 4))
    y, end, _, _ = so.conv_forward(x, w, None, None, None, 1)
    y1, mid, _, _ = so.conv_forward(x[:, :2], w, None, None, None, 1)
    y2, out, _, _ = so.conv_forward(x[:, 2:], w, None, mid, None, 1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.allclose(out, end, atol=0)


def test_oracle_catches_planted_mistakes():
    """A decay left out, a gate swapped and a tap shifted move results past the
    limits that the GPU tests use."""
    v, _, _ = _scan(5, T=40, D=8)
    y, _, _, ym, _ = so.scan_forward(v["x"], v["r"], v["i"], v["lam"], v["h0"], None, 8.0)
    wrong = so.scan_forward(v["x"], v["i"], v["r"], v["lam"], v["h0"], None, 8.0)[0]
    with pytest.raises(AssertionError):
        so.check(wrong, y, ym, 60, "bf16", "gates swapped")
    wrong = so.scan_forward(v["x"], v["r"], v["i"], v["lam"], v["h0"], None, 7.9)[0]
    with pytest.raises(AssertionError):
        so.check(wrong, y, ym, 60, "f32", "decay off")
    w = np.random.default_rng(6).normal(size=(8, 4))
    yc, _, _, um = so.conv_forward(v["x"], w, None, None, None, 0)
    wrong = so.conv_forward(v["x"], np.roll(w, 1, 1), None, None, None, 0)[0]
    with pytest.raises(AssertionError):
        so.check(wrong, yc, um, 60, "bf16", "tap shifted")
