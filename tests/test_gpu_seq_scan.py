"""The gated linear recurrence on the GPU, both directions, against the 64-bit
oracle.

Tolerances: every result is a sum of products whose factors (gates, decays,
their products over up to T tokens) each lose a few units of 2^-24, a decay
up to a few units more for each unit of its rate; so (T + 16) * (4 + 6 rate)
steps of 2^-24 of the magnitude, plus one rounding to the storage type."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import seq_oracle as so
from depthwise_convolution_forward_gb300 import inputs
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, f64, host, place, randn, same_bits

pytestmark = pytest.mark.gpu
C = 8.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(seed, B, T, D, dtype, lens=None, lam="slow", h0=True):
    g = torch.Generator().manual_seed(seed)
    s = {"x": randn(g, B, T, D, dtype=dtype), "r": randn(g, B, T, D, dtype=dtype), "i": randn(g, B, T, D, dtype=dtype),
         "dy": randn(g, B, T, D, dtype=dtype), "dhT": randn(g, B, D), "h0": randn(g, B, D) if h0 else None}
    if lam == "slow":  # slowest decay 0.9 ... 0.999
        s["lam"] = torch.log(torch.expm1(-torch.log(torch.rand(D, generator=g) * 0.099 + 0.9) / C)).to(DEV)
    else:  # rates from 1e-4 to 30: both sides of every branch on the decay
        s["lam"] = (torch.rand(D, generator=g) * 14 - 11).to(DEV)
    s["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    if lens is not None:  # what lies past a sequence's end is never read
        for b, n in enumerate(lens):
            for k in ("x", "r", "i", "dy"):
                s[k][b, max(0, min(n, T)):] = float("nan")
    return s


def run(s, dtype, strides=None, offset=0, backward=True, stream=None, h0_alias=False):
    """Forward (and backward) with guarded outputs; dict of results."""
    B, T, D = s["x"].shape
    st = strides or {}
    p = gc.make_scan_problem(B, T, D, C, *(st.get(k) for k in ("x", "r", "i", "y")))
    full = lambda k: (*st[k], 1) if k in st else None  # noqa: E731
    put = lambda t, k: place(t, full(k), offset) if k in st else t  # noqa: E731
    x, r, i, dy = put(s["x"], "x"), put(s["r"], "r"), put(s["i"], "i"), put(s["dy"], "y")
    dt = s["x"].dtype
    y, hT = Guarded((B, T, D), dt, full("y"), offset if "y" in st else 0), Guarded((B, D), torch.float32)
    saved = Guarded((gc.gconv_gated_scan_saved_size(p, code(dtype)) // 4,), torch.float32)
    h0 = s["h0"]
    if h0_alias:
        hT.t.copy_(h0)
        h0 = hT.t
    stream = stream or torch.cuda.current_stream()
    gc.gconv_gated_scan_fwd(x, r, i, s["lam"], h0, s["lens"], y.t, hT.t, saved.t if backward else None, p, code(dtype), stream)
    out = {"y": y, "hT": hT}
    if backward:
        n = gc.gconv_gated_scan_bwd_workspace_size(p, code(dtype))
        ws = Guarded((n,), torch.uint8)
        o = {k: Guarded((B, T, D), dt, full(q), offset if q in st else 0) for k, q in (("dx", "x"), ("dr", "r"), ("di", "i"))}
        o["dlam"], o["dh0"] = Guarded((D,), torch.float32), Guarded((B, D), torch.float32)
        gc.gconv_gated_scan_bwd(dy, s["dhT"], x, r, i, s["lam"], s["lens"], saved.t, o["dx"].t, o["dr"].t, o["di"].t,
                                o["dlam"].t, o["dh0"].t, p, code(dtype), ws.t, n, stream)
        out.update(o)
        stream.synchronize()
        ws.check(), saved.check()
    stream.synchronize()
    return {k: v.check() for k, v in out.items()}


def compare(s, got, dtype, backward=True):
    x, r, i, lam, h0, dy, dhT = f64(*(s[k] for k in ("x", "r", "i", "lam", "h0", "dy", "dhT")))
    lens = None if s["lens"] is None else s["lens"].cpu().numpy()
    if lens is not None:
        x, r, i, dy = (np.nan_to_num(v) for v in (x, r, i, dy))
    B, T, D = x.shape
    rate = C * so.softplus(lam).max()
    steps = (T + 16) * (4 + 6 * rate)
    y, hT, _, ym, hm = so.scan_forward(x, r, i, lam, h0, lens, C)
    so.check(host(got["y"]), y, ym, steps, dtype, "y")
    so.check(host(got["hT"]), hT, hm, steps, "f32", "hT")
    if not backward:
        return
    g, m = so.scan_backward(dy, dhT, x, r, i, lam, h0, lens, C)
    for k in ("dx", "dr", "di"):
        so.check(host(got[k]), g[k], m[k], steps, dtype, k)
    so.check(host(got["dh0"]), g["dh0"], m["dh0"], steps, "f32", "dh0")
    so.check(host(got["dlam"]), g["dlam"], m["dlam"], steps + B * T, "f32", "dlam")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 1, 64), (2, 2, 5), (1, 7, 130), (2, 16, 64), (1, 17, 33), (2, 64, 128),
                                   (1, 65, 66), (3, 127, 96), (1, 300, 256), (2, 515, 72), (1, 1100, 64)])
def test_against_oracle(dtype, B, T, D):
    s = make(10 * T + D, B, T, D, dtype)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,T", [([0, 1, 5], 5), ([16, 15, 17, 0], 40), ([100, 64, 63, 65, 128], 130),
                                    ([600, 0, 513, -3, 900], 600)])
def test_ragged(dtype, lens, T):
    """Empty sequences, lengths at every boundary, lengths outside 0 ... T; NaN past
    every end."""
    s = make(T, len(lens), T, 64, dtype, lens)
    got = run(s, dtype)
    compare(s, got, dtype)
    for b, n in enumerate(lens):
        n = max(0, min(n, T))
        for k in ("y", "dx", "dr", "di"):
            assert bool((got[k][b, n:] == 0).all()), k
        if n == 0:
            assert same_bits(got["hT"][b], s["h0"][b]) and same_bits(got["dh0"][b], s["dhT"][b])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("T,D", [(3, 40), (150, 128), (400, 61)])
def test_every_decay(dtype, T, D):
    """Rates from 1e-4 to 30: decays next to one and next to nothing."""
    s = make(7, 2, T, D, dtype, lam="wide")
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 150])
def test_no_initial_state(dtype, T):
    s = make(8, 2, T, 64, dtype, h0=False)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 40, 333])
@pytest.mark.parametrize("layout", ["sliced", "odd", "time_major"])
def test_strides(dtype, T, layout):
    """Column slices of a wider tensor, an odd pitch at an odd offset, and
    time-major order."""
    B, D = 3, 64
    st = {"sliced": {"x": (T * 3 * D, 3 * D), "r": (T * 2 * D, 2 * D), "i": (T * 3 * D, 3 * D)},
          "odd": {k: (T * (D + 5) + 3, D + 5) for k in ("x", "r", "i", "y")},
          "time_major": {k: (D, B * D) for k in ("x", "r", "i", "y")}}[layout]
    s = make(T, B, T, D, dtype)
    compare(s, run(s, dtype, st, 1 if layout == "odd" else 0), dtype)


def test_slices_of_one_projection():
    """x, r, i (and their gradients) as column slices of one buffer each."""
    B, T, D = 2, 70, 64
    s = make(3, B, T, D, "bf16")
    wide = torch.cat([s["x"], s["r"], s["i"]], 2).contiguous()
    st = (T * 3 * D, 3 * D)
    p = gc.make_scan_problem(B, T, D, C, st, st, st)
    c = code("bf16")
    y, hT = torch.empty_like(s["x"]), torch.empty_like(s["h0"])
    saved = torch.empty(gc.gconv_gated_scan_saved_size(p, c), dtype=torch.uint8, device=DEV)
    n = gc.gconv_gated_scan_bwd_workspace_size(p, c)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    q = torch.cuda.current_stream()
    x, r, i = wide[..., :D], wide[..., D:2 * D], wide[..., 2 * D:]
    gc.gconv_gated_scan_fwd(x, r, i, s["lam"], s["h0"], None, y, hT, saved, p, c, q)
    d = torch.full_like(wide, float("nan"))
    dlam, dh0 = torch.empty_like(s["lam"]), torch.empty_like(s["h0"])
    gc.gconv_gated_scan_bwd(s["dy"], s["dhT"], x, r, i, s["lam"], None, saved, d[..., :D], d[..., D:2 * D], d[..., 2 * D:],
                            dlam, dh0, p, c, ws, n, q)
    compare(s, {"y": y, "hT": hT, "dx": d[..., :D], "dr": d[..., D:2 * D], "di": d[..., 2 * D:], "dlam": dlam, "dh0": dh0},
            "bf16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gates_at_their_ends(dtype):
    """Gates of +-infinity and large values, on slow and fast channels: finite
    results, the limits of the formulas."""
    B, T, D = 1, 40, 64
    s = make(9, B, T, D, dtype)
    big = torch.tensor([float("inf"), float("-inf"), 90.0, -90.0, 30.0, -30.0], device=DEV).to(s["x"].dtype)
    s["r"][0, 5:35] = big.repeat(5)[:, None]
    s["i"][0, 5:35] = big.repeat_interleave(5)[:, None]
    got = run(s, dtype)
    compare(s, got, dtype)


def test_state_in_place_and_token_by_token():
    """A sequence decoded one token at a time in place is the whole sequence,
    to the bit of the state's fp32 steps at T = 1 and within the tolerance of the scan."""
    B, T, D = 2, 23, 96
    s = make(4, B, T, D, "f32")
    whole = run(s, "f32", backward=False, h0_alias=True)
    h = s["h0"].clone()
    p = gc.make_scan_problem(B, 1, D, C)
    ys = []
    for t in range(T):
        y = torch.empty(B, 1, D, device=DEV)
        gc.gconv_gated_scan_fwd(s["x"][:, t].contiguous(), s["r"][:, t].contiguous(), s["i"][:, t].contiguous(), s["lam"], h,
                                None, y, h, None, p, code("f32"), torch.cuda.current_stream())
        ys.append(y)
    torch.cuda.synchronize()
    compare(s, {"y": torch.cat(ys, 1), "hT": h}, "f32", backward=False)
    compare(s, whole, "f32", backward=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_carry_gradients(dtype):
    """Backward through two parts, the second's dh0 feeding the first's dhT,
    against the oracle's whole."""
    B, T, D, cut = 2, 90, 64, 37
    s = make(5, B, T, D, dtype)
    first = {k: (v[:, :cut].contiguous() if k in ("x", "r", "i", "dy") else v) for k, v in s.items()}
    mid = run(first, dtype, backward=False)["hT"]
    second = {k: (v[:, cut:].contiguous() if k in ("x", "r", "i", "dy") else v) for k, v in s.items()}
    second["h0"] = mid
    b = run(second, dtype)
    first["dhT"] = b["dh0"]
    a = run(first, dtype)
    got = {k: torch.cat([a[k], b[k]], 1) for k in ("y", "dx", "dr", "di")}
    got.update(hT=b["hT"], dh0=a["dh0"], dlam=a["dlam"] + b["dlam"])
    compare(s, got, dtype)


def test_gradient_against_differences():
    """The loss's slope along a random direction, from the kernel's own forward
    in fp32, against its gradients.  With a step of 2^-6 the truncation is below
    1e-3 of the slope's magnitude and the rounding of the loss (2^-24 of its
    magnitude over the step) below 1e-4."""
    B, T, D = 2, 33, 64
    s = make(6, B, T, D, "f32")
    got = run(s, "f32")
    g = torch.Generator().manual_seed(60)
    eps = 2.0 ** -6
    for name, key in (("x", "dx"), ("r", "dr"), ("i", "di"), ("lam", "dlam"), ("h0", "dh0")):
        v = randn(g, *s[name].shape, std=1.0)

        def loss(sign):
            out = run({**s, name: s[name] + sign * eps * v}, "f32", backward=False)
            return (out["y"].double() * s["dy"].double()).sum() + (out["hT"].double() * s["dhT"].double()).sum()

        slope = float((loss(1) - loss(-1)) / (2 * eps))
        want = float((got[key].double() * v.double()).sum())
        size = float((got[key].double() * v.double()).abs().sum())
        assert abs(slope - want) <= 2e-3 * size, (name, slope, want, size)


def test_deterministic_and_on_another_stream():
    s = make(11, 4, 300, 128, "bf16")
    a = run(s, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = run(s, "bf16", stream=st)
    for k in a:
        assert same_bits(a[k], b[k]), k


def test_graph_replay_on_new_inputs():
    B, T, D = 2, 130, 64
    s, other = make(12, B, T, D, "bf16"), make(13, B, T, D, "bf16")
    p, c = gc.make_scan_problem(B, T, D, C), code("bf16")
    y, hT = torch.empty_like(s["x"]), torch.empty_like(s["h0"])
    saved = torch.empty(gc.gconv_gated_scan_saved_size(p, c), dtype=torch.uint8, device=DEV)
    n = gc.gconv_gated_scan_bwd_workspace_size(p, c)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    o = {k: torch.empty_like(s["x"]) for k in ("dx", "dr", "di")}
    o["dlam"], o["dh0"] = torch.empty_like(s["lam"]), torch.empty_like(s["h0"])
    s["lam"].copy_(other["lam"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q = torch.cuda.current_stream()
        gc.gconv_gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["h0"], None, y, hT, saved, p, c, q)
        gc.gconv_gated_scan_bwd(s["dy"], s["dhT"], s["x"], s["r"], s["i"], s["lam"], None, saved, o["dx"], o["dr"], o["di"],
                                o["dlam"], o["dh0"], p, c, ws, n, q)
    for k in ("x", "r", "i", "dy", "dhT", "h0"):
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    compare(other, {"y": y, "hT": hT, **o}, "bf16")


def test_offsets_past_32_bits():
    """Sequences that start more than 2^31 elements apart."""
    B, T, D = 2, 50, 64
    far = (1 << 31) + 64
    s = make(14, B, T, D, "bf16")
    x, y = (torch.empty(far + T * D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    xv, yv = (t.as_strided((B, T, D), (far, D, 1)) for t in (x, y))
    xv.copy_(s["x"])
    p, c = gc.make_scan_problem(B, T, D, C, x_stride=(far, D), y_stride=(far, D)), code("bf16")
    hT = torch.empty_like(s["h0"])
    gc.gconv_gated_scan_fwd(xv, s["r"], s["i"], s["lam"], s["h0"], None, yv, hT, None, p, c, torch.cuda.current_stream())
    torch.cuda.synchronize()
    compare(s, {"y": yv, "hT": hT}, "bf16", backward=False)


def test_a_long_sequence():
    """Many blocks along time: the carried state over 20,000 tokens, against the
    oracle at the end and over the whole output."""
    B, T, D = 1, 20000, 64
    s = make(15, B, T, D, "bf16")
    compare(s, run(s, "bf16", backward=False), "bf16", backward=False)


def test_many_channels_and_sequences():
    s = make(16, 9, 70, 1000, "f16")
    compare(s, run(s, "f16"), "f16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 192), (100, 192), (61, 95)])
def test_channels_of_every_kind(dtype, T, D):
    """Neighbouring groups of 32 channels with rates up to 0.1, up to 9, near
    1e-12 and near 40: whole warps of each kind, and warps that hold two."""
    s = make(11, 2, T, D, dtype)
    lam = s["lam"]
    u = torch.rand(D, generator=torch.Generator().manual_seed(12)).to(DEV)
    kind = torch.arange(D, device=DEV) // 32 % 6
    lam = torch.where(kind == 1, u * 4 - 3.3, lam)
    lam = torch.where((kind == 2) | (kind == 3), u - 30, lam)
    s["lam"] = torch.where(kind == 5, u + 5, lam)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_sequence_for_each_block(dtype):
    """Sequences enough that no two blocks share one, long and ragged ones."""
    B, T = 80, 1030
    lens = [T - 13 * k if k % 7 else k // 7 * 48 for k in range(B)]
    s = make(13, B, T, 64, dtype, lens)
    got = run(s, dtype)
    compare(s, got, dtype)
    for k in ("y", "dx", "dr", "di"):
        assert all(bool((got[k][b, n:] == 0).all()) for b, n in enumerate(lens)), k
