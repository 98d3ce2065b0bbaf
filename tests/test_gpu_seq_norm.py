"""Residual + RMS norm to 8 bits, and the row quantiser, on the GPU.

Tolerances: the sum of D squares in fp32 loses at most D + 8 steps of 2^-24
(half of that in its root); a quantised value's argument loses a few more, so q
is within 0.5 + 127 * 16 * 2^-24 of the exact quotient."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import seq_oracle as so
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, host, place, randn, same_bits

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(seed, M, D, dtype):
    g = torch.Generator().manual_seed(seed)
    return {"x": randn(g, M, D, dtype=dtype), "res": randn(g, M, D, dtype=dtype, std=2.0),
            "w": (torch.rand(D, generator=g) + 0.5).to(DEV).to(randn(g, 1, dtype=dtype).dtype)}


def run(s, dtype, res=True, weight=True, want="yq", alias=None, strides=(0, 0, 0), offset=0, eps=EPS):
    M, D = s["x"].shape
    p = gc.make_norm_problem(M, D, eps, *strides)
    st = [(v, 1) if v else None for v in strides]
    off = [offset if v else 0 for v in st]
    x = place(s["x"], st[0], off[0]) if st[0] else s["x"].clone()
    r = (place(s["res"], st[1], off[1]) if st[1] else s["res"].clone()) if res else None
    dt = x.dtype
    ro = Guarded((M, D), dt, st[1], off[1])
    ro_t = {"x": x, "res": r}.get(alias, ro.t)
    y = Guarded((M, D), dt, st[2], off[2]) if "y" in want else None
    q = Guarded((M, D), torch.int8) if "q" in want else None
    sc = Guarded((M,), torch.float32) if "q" in want else None
    gc.gconv_rms_norm_q8(x, r, s["w"] if weight else None, ro_t, y and y.t, q and q.t, sc and sc.t, p, code(dtype),
                         torch.cuda.current_stream())
    torch.cuda.synchronize()
    out = {"res": ro_t.clone() if alias else ro.check()}
    for k, v in (("y", y), ("q", q), ("scale", sc)):
        if v is not None:
            out[k] = v.check()
    return out


def compare(s, got, dtype, res=True, weight=True, eps=EPS):
    h = (s["x"].float() + s["res"].float()).to(s["x"].dtype) if res else s["x"]
    assert same_bits(got["res"], h)
    M, D = h.shape
    w = host(s["w"]) if weight else np.ones(D)
    v, scale = so.norm_rows(host(h), w, eps)
    if "y" in got:
        so.check(host(got["y"]), v, np.abs(v), D / 2 + 16, dtype, "y")
    if "q" in got:
        so.check(host(got["scale"]), scale, scale, D / 2 + 16, "f32", "scale")
        want = np.divide(v, scale[:, None], out=np.zeros_like(v), where=scale[:, None] > 0)
        assert np.abs(host(got["q"]) - want).max() <= 0.5 + 127 * 16 * so.U


SHAPES = [(1, 1), (3, 7), (2, 32), (5, 64), (4, 100), (2, 256), (3, 520), (7, 1024), (2, 2047), (3, 2048), (2, 4096),
          (2, 5000), (1, 8192), (2, 8200), (1, 16384), (1, 32768),
          (1501, 64), (701, 256), (650, 512), (703, 1016), (640, 1032)]  # many rows: a warp or a block a row


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,D", SHAPES)
def test_against_oracle(dtype, M, D):
    s = make(M + D, M, D, dtype)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("want", ["y", "q"])
def test_optional_parts(dtype, res, weight, want):
    s = make(2, 5, 512, dtype)
    compare(s, run(s, dtype, res, weight, want), dtype, res, weight)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("alias", ["x", "res"])
@pytest.mark.parametrize("D", [77, 1024])
def test_residual_in_place(dtype, alias, D):
    s = make(3, 6, D, dtype)
    compare(s, run(s, dtype, alias=alias), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("strides,offset", [((512, 0, 0), 0), ((264, 320, 288), 8), ((259, 301, 263), 1)])
def test_strides(dtype, strides, offset):
    s = make(4, 9, 256, dtype)
    compare(s, run(s, dtype, strides=strides, offset=offset), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [40, 1024, 9001])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rows_at_the_ends(dtype, D, eps):
    """A row of zeros, rows with one NaN and one infinity, tiny and large rows,
    beside ordinary ones."""
    s = make(5, 7, D, dtype)
    tiny = {"f32": 1e-38, "f16": 6e-8, "bf16": 1e-38}[dtype]
    big = {"f32": 1e17, "f16": 2e4, "bf16": 1e17}[dtype]
    s["x"][1], s["res"][1] = 0, 0
    s["x"][2, D // 2], s["x"][3, D - 1] = float("nan"), float("inf")
    s["x"][4], s["res"][4] = tiny, 0
    s["x"][5] = s["x"][5] * (big / 8)
    s["res"][5] = 0
    got = run(s, dtype, eps=eps)
    q, scale = host(got["q"]), host(got["scale"])
    assert scale[1] == 0 and not q[1].any() and not host(got["y"])[1].any()
    assert np.isnan(scale[2:4]).all() and not q[2:4].any()
    rows = [0, 5, 6] + ([4] if eps else [])
    sub = {k: v[rows] if k != "w" else v for k, v in s.items()}
    compare(sub, {k: v[rows] for k, v in got.items()}, dtype, eps=eps)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,D", [(3, 1), (5, 64), (2, 100), (4, 2048), (3, 7777)])
def test_quantize_rows(dtype, M, D):
    s = make(6, M, D, dtype)
    x = s["x"]
    if M > 2 and D > 1:
        x[0] = 0
        x[1] *= 1e-4
    q, sc = Guarded((M, D), torch.int8), Guarded((M,), torch.float32)
    gc.gconv_quantize_rows_q8(x, q.t, sc.t, gc.make_norm_problem(M, D), code(dtype), torch.cuda.current_stream())
    q, sc = host(q.check()), host(sc.check())
    v = host(x)
    scale = np.abs(v).max(1) / 127
    so.check(sc, scale, scale, 4, "f32", "scale")
    want = np.divide(v, scale[:, None], out=np.zeros_like(v), where=scale[:, None] > 0)
    assert np.abs(q - want).max() <= 0.5 + 127 * 16 * so.U and np.abs(q).max() <= 127


def test_quantize_rows_of_tiny_values():
    """Rows whose 127 / max|x| passes fp32."""
    x = torch.tensor([[1e-38, -2e-38, 5e-39, 0.0], [3e-40, -1e-40, 0.0, 1e-40]], device=DEV)
    q, sc = torch.empty(2, 4, dtype=torch.int8, device=DEV), torch.empty(2, device=DEV)
    gc.gconv_quantize_rows_q8(x, q, sc, gc.make_norm_problem(2, 4), code("f32"), torch.cuda.current_stream())
    assert q[0].tolist() == [64, -127, 32, 0] or q[0].tolist() == [63, -127, 32, 0]
    assert q[1].tolist() == [127, -42, 0, 42]


def test_no_rows():
    p = gc.make_norm_problem(0, 64)
    x = torch.empty(0, 64, device=DEV)
    q, sc = torch.empty(0, 64, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)
    gc.gconv_rms_norm_q8(x, None, None, None, None, 16, 16, p, code("f32"), None)
    gc.gconv_quantize_rows_q8(16, 16, 16, p, code("f32"), None)


def test_deterministic_and_on_another_stream():
    s = make(8, 100, 1536, "bf16")
    a = run(s, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = run(s, "bf16")
    for k in a:
        assert same_bits(a[k], b[k])


def test_graph_replay():
    s, other = make(9, 17, 640, "f16"), make(10, 17, 640, "f16")
    ro, q, sc = torch.empty_like(s["x"]), torch.empty(17, 640, dtype=torch.int8, device=DEV), torch.empty(17, device=DEV)
    p = gc.make_norm_problem(17, 640, EPS)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gc.gconv_rms_norm_q8(s["x"], s["res"], s["w"], ro, None, q, sc, p, code("f16"), torch.cuda.current_stream())
    for k in s:
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    compare(other, {"res": ro, "q": q, "scale": sc}, "f16")


def quotients(f):
    """127 f / max|f| to the nearest integer, ties to even: exact for f of up to 24
    bits, whose quotient lies at a tie or 2^-25 away from it."""
    m = np.abs(f).max(1, keepdims=True)
    return np.rint(np.divide(127 * f, m, out=np.zeros_like(f), where=m > 0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [100, 101, 512, 2048, 4096])
@pytest.mark.parametrize("M", [9, 700])
def test_ties_go_to_even(dtype, D, M):
    """Rows whose quotients are all halves, for every weight of eight bits: 127 c at
    the row's largest, (k + 1/2) c elsewhere."""
    k = torch.arange(M * D, dtype=torch.float32).reshape(M, D) % 254 - 127 + 0.5
    k[:, 3] = 127
    x = k.to(DEV).to(randn(torch.Generator(), 1, dtype=dtype).dtype)
    for c in (1.0, 3.0, 131.0, 149.0, 171.0, 197.0, 253.0):
        s = {"x": x, "res": torch.zeros_like(x), "w": torch.full((D,), c / 128, device=DEV).to(x.dtype)}
        got = run(s, dtype, want="q")
        assert np.array_equal(host(got["q"]), quotients(host(x)))
        q, sc = torch.empty(M, D, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
        v = x.float() * c / 128  # fp32 rows that need the weight's bits as well
        gc.gconv_quantize_rows_q8(v, q, sc, gc.make_norm_problem(M, D), code("f32"), torch.cuda.current_stream())
        assert np.array_equal(host(q), quotients(host(x)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,D", [(16, 2048), (300, 4096), (2000, 1001), (3000, 512)])
def test_nearest_values(dtype, M, D):
    """Every 8-bit value is the nearest one, of h weight as fp32 holds it: always where
    that takes up to 16 bits, as in bf16; within 2^-24 of a tie, which is more than the
    roundings of a quotient's distance from its integer add up to, either side where
    it takes more."""
    s = make(15, M, D, dtype)
    for weight in (True, False):
        got = run(s, dtype, want="q", weight=weight)
        f = (s["x"].float() + s["res"].float()).to(s["x"].dtype).float()
        f = host(f * s["w"].float() if weight else f)
        if dtype == "bf16" or (dtype == "f16" and not weight):
            assert np.array_equal(host(got["q"]), quotients(f))
        assert np.abs(host(got["q"]) - 127 * f / np.abs(f).max(1, keepdims=True)).max() <= 0.5 + 2.0 ** -24


def test_two_threads_with_rows_of_different_widths():
    """Rows that need more shared memory than the default, of two widths, from two
    threads and streams."""
    import threading

    widths = [32767, 16385, 13001]
    xs = [make(14, 3, D, "f32")["x"] for D in widths]
    errors, got = [], {}
    gate = threading.Barrier(len(widths))

    def work(x):
        M, D = x.shape
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            q, sc, p = torch.empty(M, D, dtype=torch.int8, device=DEV), torch.empty(M, device=DEV), gc.make_norm_problem(M, D)
            gate.wait(30)
            for _ in range(3000):
                gc.gconv_quantize_rows_q8(x, q, sc, p, code("f32"), st)
            st.synchronize()
            got[D] = q, sc
        except Exception as e:  # noqa: BLE001
            errors.append(f"{D}: {e}")

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(x,)) for x in xs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for x in xs:
        q, sc = got[x.shape[1]]
        scale = np.abs(host(x)).max(1) / 127
        so.check(host(sc), scale, scale, 4, "f32", "scale")
        assert np.abs(host(q) - host(x) / scale[:, None]).max() <= 0.5 + 127 * 16 * so.U


@pytest.mark.parametrize("dtype,D", [("f32", 12224), ("f32", 12225), ("f32", 12256), ("f32", 12288), ("f32", 12289),
                                     ("f16", 24448), ("bf16", 24456), ("bf16", 24575), ("f16", 24576), ("bf16", 24577)])
def test_widths_about_the_default_shared_memory(dtype, D):
    """Rows that fill a block's default 48 KB of shared memory, beside the few bytes
    that the kernel has of its own."""
    s = make(16, 3, D, dtype)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 40, 512, 1024, 9001, 16384])
@pytest.mark.parametrize("M", [9, 700])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-33, 1e-30, 1e-5])
def test_rows_whose_squares_pass_fp32(dtype, D, M, weight, eps):
    """Rows down to the smallest numbers, with eps = 0, where v is of order 1, and with
    ones beside and above their squares: those need more range than fp32 has, the
    result does not."""
    if D > 1024 and M > 9:
        M = 21
    s = make(13, M, D, dtype)
    size = torch.tensor([1e-15, 1e-18, 1e-20, 1e-24, 1e-30, 1e-36, 1e-38, 3e-40, 1.0])[torch.arange(M) % 9].to(DEV)
    s["x"] = (s["x"].double() * size.double()[:, None]).to(s["x"].dtype)
    s["res"] = torch.zeros_like(s["x"])
    s["res"][0] = s["x"][0]
    # a value may vanish in the type: keep one in every row
    s["x"][:, D // 2] = torch.where(s["x"][:, D // 2] == 0, size.to(s["x"].dtype), s["x"][:, D // 2])
    got = run(s, dtype, weight=weight, eps=eps)
    h = (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    assert same_bits(got["res"], h)
    # eps as fp32 holds it; the factor and the sum lose what `compare` allows, the smallest scales 2^-149
    w = host(s["w"]) if weight else np.ones(D)
    v, scale = so.norm_rows(host(h), w, float(np.float32(eps)))
    so.check(host(got["y"]), v, np.abs(v), D / 2 + 16, dtype, "y")
    assert np.all(np.abs(host(got["scale"]) - scale) <= (D / 2 + 18) * so.U * scale + 2.0 ** -149)
    want = v / scale[:, None]
    assert np.abs(host(got["q"]) - want).max() <= 0.5 + 127 * 16 * so.U
