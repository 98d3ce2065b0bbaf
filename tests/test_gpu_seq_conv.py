"""The causal depthwise convolution on the GPU against the 64-bit oracle.

Tolerances: a pre-activation is a sum of K products and a bias in fp32 (K + 4
steps of 2^-24 of its magnitude); SiLU's slope is at most 1.1 and its logistic
function loses a few units plus one for each unit of |u|; the backward pass's
sums over tokens add one step a token."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import seq_oracle as so
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, f64, host, place, randn, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(seed, B, T, D, K, dtype, lens=None, state=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    s = {"x": randn(g, B, T, D, dtype=dtype), "dy": randn(g, B, T, D, dtype=dtype), "w": randn(g, D, K, dtype=dtype, std=0.5),
         "bias": randn(g, D, dtype=dtype, std=0.1) if bias else None,
         "state": randn(g, B, K - 1, D, dtype=dtype) if state else None,
         "dstate_out": randn(g, B, K - 1, D, dtype=dtype) if state else None,
         "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if lens is not None:
        for b, n in enumerate(lens):
            for k in ("x", "dy"):
                s[k][b, max(0, min(n, T)):] = float("nan")
    return s


def run(s, dtype, act, strides=None, offset=0, backward=True, stream=None):
    B, T, D = s["x"].shape
    K = s["w"].shape[1]
    st = strides or {}
    p = gc.make_conv1d_problem(B, T, D, K, act, st.get("x"), st.get("y"))
    full = lambda k: (*st[k], 1) if k in st else None  # noqa: E731
    x = place(s["x"], full("x"), offset) if "x" in st else s["x"]
    dy = place(s["dy"], full("y"), offset) if "y" in st else s["dy"]
    dt = s["x"].dtype
    stream = stream or torch.cuda.current_stream()
    o = {"y": Guarded((B, T, D), dt, full("y"), offset if "y" in st else 0), "state": Guarded((B, K - 1, D), dt)}
    gc.gconv_causal_conv1d_fwd(x, s["w"], s["bias"], s["state"], s["lens"], o["y"].t, o["state"].t, p, code(dtype), stream)
    if backward:
        n = gc.gconv_causal_conv1d_bwd_workspace_size(p, code(dtype))
        ws = Guarded((n,), torch.uint8)
        o["dx"], o["dw"] = Guarded((B, T, D), dt, full("x"), offset if "x" in st else 0), Guarded((D, K), dt)
        o["dbias"], o["dstate"] = Guarded((D,), dt), Guarded((B, K - 1, D), dt)
        gc.gconv_causal_conv1d_bwd(dy, s["dstate_out"], x, s["w"], s["bias"], s["state"], s["lens"], o["dx"].t, o["dw"].t,
                                   o["dbias"].t, o["dstate"].t, p, code(dtype), ws.t, n, stream)
        stream.synchronize()
        ws.check()
    stream.synchronize()
    return {k: v.check() for k, v in o.items()}


def compare(s, got, dtype, act, backward=True):
    x, w, bias, state, dy, ds = f64(*(s[k] for k in ("x", "w", "bias", "state", "dy", "dstate_out")))
    lens = None if s["lens"] is None else s["lens"].cpu().numpy()
    if lens is not None:
        x, dy = np.nan_to_num(x), np.nan_to_num(dy)
    B, T, D = x.shape
    K = w.shape[1]
    y, out, u, um = so.conv_forward(x, w, bias, state, lens, act)
    top = np.abs(u).max() if u.size else 0
    so.check(host(got["y"]), y, um, 1.1 * (K + 4) + 16 + 2 * top, dtype, "y")
    assert np.array_equal(host(got["state"]), out)
    if not backward:
        return
    g, m = so.conv_backward(dy, ds, x, w, bias, state, lens, act)
    steps = 4 * (K + 4) + 16 + 4 * top
    for k in ("dx", "dstate"):
        so.check(host(got[k]), g[k], m[k], steps, dtype, k)
    for k in ("dw", "dbias"):
        so.check(host(got[k]), g[k], m[k], steps + B * T, dtype, k)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("B,T,D,K", [(1, 1, 1, 1), (2, 1, 64, 4), (3, 2, 8, 4), (1, 3, 7, 2), (2, 5, 33, 3), (1, 9, 64, 8),
                                     (2, 40, 130, 5), (1, 64, 256, 4), (2, 131, 72, 4), (1, 300, 16, 7), (2, 200, 264, 2)])
def test_against_oracle(dtype, act, B, T, D, K):
    s = make(T + D, B, T, D, K, dtype)
    compare(s, run(s, dtype, act), dtype, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("lens,T", [([0, 1, 2, 3], 3), ([16, 15, 17, 0, 1], 33), ([100, 64, 0, 63, 65, 128, 2, -1, 999], 130)])
def test_ragged(dtype, K, lens, T):
    """Sequences shorter than the filter, empty ones, lengths at boundaries and
    outside 0 ... T; NaN past every end."""
    s = make(T + K, len(lens), T, 64, K, dtype, lens)
    got = run(s, dtype, 1)
    compare(s, got, dtype, 1)
    for b, n in enumerate(lens):
        n = max(0, min(n, T))
        assert bool((got["y"][b, n:] == 0).all()) and bool((got["dx"][b, n:] == 0).all())
        if n == 0:
            assert same_bits(got["state"][b], s["state"][b]) and same_bits(got["dstate"][b], s["dstate_out"][b])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("bias", [False, True])
def test_without_state(dtype, bias):
    s = make(3, 2, 50, 64, 4, dtype, state=False, bias=bias)
    compare(s, run(s, dtype, 1), dtype, 1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 70])
@pytest.mark.parametrize("layout", ["sliced", "odd", "time_major"])
def test_strides(dtype, T, layout):
    B, D = 3, 64
    st = {"sliced": {"x": (T * 3 * D, 3 * D)}, "odd": {k: (T * (D + 5) + 3, D + 5) for k in ("x", "y")},
          "time_major": {k: (D, B * D) for k in ("x", "y")}}[layout]
    s = make(T, B, T, D, 4, dtype)
    compare(s, run(s, dtype, 1, st, 1 if layout == "odd" else 0), dtype, 1)


def test_nothing_outside_the_filter_is_read():
    """A NaN reaches the outputs whose filter covers it, and no others."""
    s = make(5, 1, 64, 64, 3, "f32")
    s["x"][0, 20] = float("nan")
    p = gc.make_conv1d_problem(1, 64, 64, 3, 0)
    y = torch.empty_like(s["x"])
    gc.gconv_causal_conv1d_fwd(s["x"], s["w"], s["bias"], s["state"], None, y, None, p, code("f32"), torch.cuda.current_stream())
    bad = torch.isnan(y).all(2)[0].cpu()
    assert bad[20:23].all() and not torch.isnan(y[0, :20]).any() and not torch.isnan(y[0, 23:]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_token_by_token_in_place(dtype):
    """One token at a time with the state in place is the whole sequence."""
    B, T, D, K = 3, 11, 72, 4
    s = make(6, B, T, D, K, dtype)
    state = s["state"].clone()
    p = gc.make_conv1d_problem(B, 1, D, K, 1)
    ys = []
    for t in range(T):
        y = torch.empty(B, 1, D, dtype=s["x"].dtype, device=DEV)
        gc.gconv_causal_conv1d_fwd(s["x"][:, t].contiguous(), s["w"], s["bias"], state, None, y, state, p, code(dtype),
                                   torch.cuda.current_stream())
        ys.append(y)
    torch.cuda.synchronize()
    compare(s, {"y": torch.cat(ys, 1), "state": state}, dtype, 1, backward=False)


def test_state_in_place_over_a_long_call():
    """state_out == state_in with many blocks along time, ragged."""
    lens = [200, 0, 1, 2, 130]
    s = make(7, 5, 200, 64, 4, "bf16", lens)
    state = s["state"].clone()
    p = gc.make_conv1d_problem(5, 200, 64, 4, 1)
    y = torch.empty_like(s["x"])
    gc.gconv_causal_conv1d_fwd(s["x"], s["w"], s["bias"], state, s["lens"], y, state, p, code("bf16"), torch.cuda.current_stream())
    torch.cuda.synchronize()
    compare(s, {"y": y, "state": state}, "bf16", 1, backward=False)


def test_gradient_against_differences():
    """As for the scan: a central difference of the kernel's own forward."""
    s = make(8, 2, 30, 64, 4, "f32")
    got = run(s, "f32", 1)
    g = torch.Generator().manual_seed(80)
    eps = 2.0 ** -6
    for name, key in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("state", "dstate")):
        v = randn(g, *s[name].shape)

        def loss(sign):
            out = run({**s, name: s[name] + sign * eps * v}, "f32", 1, backward=False)
            return (out["y"].double() * s["dy"].double()).sum() + (out["state"].double() * s["dstate_out"].double()).sum()

        slope = float((loss(1) - loss(-1)) / (2 * eps))
        want = float((got[key].double() * v.double()).sum())
        size = float((got[key].double() * v.double()).abs().sum())
        assert abs(slope - want) <= 2e-3 * size, (name, slope, want, size)


def test_optional_gradients_and_determinism():
    s = make(9, 3, 150, 72, 4, "bf16")
    a, b = run(s, "bf16", 1), run(s, "bf16", 1)
    for k in a:
        assert same_bits(a[k], b[k]), k
    p = gc.make_conv1d_problem(3, 150, 72, 4, 1)
    n = gc.gconv_causal_conv1d_bwd_workspace_size(p, code("bf16"))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    gc.gconv_causal_conv1d_bwd(s["dy"], s["dstate_out"], s["x"], s["w"], s["bias"], s["state"], None, dx, dw, None, None, p,
                               code("bf16"), ws, n, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert same_bits(dx, a["dx"]) and same_bits(dw, a["dw"])


def test_graph_replay_and_stream():
    s, other = make(10, 2, 90, 64, 4, "f16"), make(11, 2, 90, 64, 4, "f16")
    p = gc.make_conv1d_problem(2, 90, 64, 4, 1)
    y, st = torch.empty_like(s["x"]), torch.empty_like(s["state"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gc.gconv_causal_conv1d_fwd(s["x"], s["w"], s["bias"], s["state"], None, y, st, p, code("f16"), torch.cuda.current_stream())
    for k in ("x", "w", "bias", "state"):
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    compare(other, {"y": y, "state": st}, "f16", 1, backward=False)


def test_offsets_past_32_bits():
    B, T, D = 2, 40, 64
    far = (1 << 31) + 64
    s = make(12, B, T, D, 4, "bf16")
    x, y = (torch.empty(far + T * D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    xv, yv = (t.as_strided((B, T, D), (far, D, 1)) for t in (x, y))
    xv.copy_(s["x"])
    p = gc.make_conv1d_problem(B, T, D, 4, 1, (far, D), (far, D))
    st = torch.empty_like(s["state"])
    gc.gconv_causal_conv1d_fwd(xv, s["w"], s["bias"], s["state"], None, yv, st, p, code("bf16"), torch.cuda.current_stream())
    torch.cuda.synchronize()
    compare(s, {"y": yv, "state": st}, "bf16", 1, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 61])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_past_the_end_are_zero_whatever_the_weights(dtype, D, act, bad):
    lens = [40, 0, 1, 33, 128]
    s = make(15, 5, 130, D, 4, dtype, lens)
    s["w"][3, 1] = bad
    got = run(s, dtype, act)
    for b, n in enumerate(lens):
        assert bool((got["y"][b, n:] == 0).all()) and bool((got["dx"][b, n:] == 0).all())
