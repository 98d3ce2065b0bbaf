"""The 8-bit matrix product on the GPU.

Tolerances: products are exact; a sum of K of them in 32 bits loses at most K
steps of 2^-23 of the sum of their sizes (nothing while it stays below 2^24),
the scales and the bias a few steps."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import seq_oracle as so
from depthwise_convolution_forward_gb300 import inputs
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, host, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make(seed, M, N, K, dtype, top=127, bias=True):
    g = torch.Generator().manual_seed(seed)
    return {"x": torch.randint(-top - 1 if top == 127 else -top, top + 1, (M, K), generator=g).to(torch.int8).to(DEV),
            "w": torch.randint(-top - 1 if top == 127 else -top, top + 1, (N, K), generator=g).to(torch.int8).to(DEV),
            "sx": (torch.rand(M, generator=g) * 0.02 + 0.01).to(DEV), "sw": ((torch.rand(N, generator=g) + 0.5) / 64).to(DEV),
            "b": torch.randn(N, generator=g).to(inputs.DTYPES[dtype]).to(DEV) if bias else None}


def run(s, dtype, y_stride=0, offset=0):
    (M, K), N = s["x"].shape, s["w"].shape[0]
    y = Guarded((M, N), inputs.DTYPES[dtype], (y_stride, 1) if y_stride else None, offset)
    gc.gconv_matmul_q8(s["x"], s["sx"], s["w"], s["sw"], s["b"], y.t, gc.make_matmul_q8_problem(M, N, K, y_stride),
                       code(dtype), torch.cuda.current_stream())
    return y.check()


def oracle(s):
    x, w, sx, sw = (host(s[k]) for k in ("x", "w", "sx", "sw"))
    b = 0 if s["b"] is None else host(s["b"])
    scale = sx[:, None] * sw
    return (x @ w.T) * scale + b, (np.abs(x) @ np.abs(w).T) * scale, np.abs((x @ w.T) * scale) + np.abs(b)


def compare(s, got, dtype):
    K = s["x"].shape[1]
    y, sums, mag = oracle(s)
    so.check(host(got), y, mag + sums * (2 * K / 8.0 if K * 2 ** 14 > 2 ** 24 else 0), 8, dtype, "y")


# (tile widths 16 ... 160 of the tensor-core kernel, one and several tiles a block)
SHAPES = [(1280, 7680, 160), (2100, 3000, 128), (1500, 4000, 320), (700, 5000, 192), (1, 1, 1), (1, 64, 64), (2, 100, 33), (4, 256, 128), (5, 130, 512), (8, 64, 1000), (9, 65, 64), (16, 128, 256),
          (17, 200, 80), (33, 96, 144), (64, 64, 64), (100, 300, 96), (128, 128, 128), (129, 257, 160), (197, 500, 2048),
          (256, 512, 272), (300, 1000, 48), (257, 129, 1040), (1, 5000, 2048), (7, 1200, 4096)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_against_oracle(dtype, M, N, K):
    s = make(M + N + K, M, N, K, dtype)
    if dtype == "f16":
        s["sw"] /= 64  # keep sums inside the type's range
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("M,N,K", [(3, 70, 96), (8, 128, 1024), (40, 200, 1024), (200, 300, 2048), (512, 256, 512)])
def test_small_integers_are_exact(M, N, K):
    """Sums below 2^24 carry no rounding at all on either path."""
    s = make(1, M, N, K, "f32", top=7, bias=False)
    s["sx"].fill_(1.0), s["sw"].fill_(1.0)
    assert np.array_equal(host(run(s, "f32")), oracle(s)[0])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,stride,offset", [(4, 64, 128, 200, 0), (150, 136, 128, 152, 8), (150, 133, 96, 139, 1),
                                                 (2, 77, 64, 81, 3)])
def test_output_strides(dtype, M, N, K, stride, offset):
    s = make(2, M, N, K, dtype)
    compare(s, run(s, dtype, stride, offset), dtype)


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_unaligned_operands(M, shift):
    """Operands that start off a 16-byte boundary."""
    s = make(3, M, 96, 128, "f32")
    for k in ("x", "w"):
        buf = torch.empty(s[k].numel() + shift, dtype=torch.int8, device=DEV)
        v = buf[shift:].view(s[k].shape)
        v.copy_(s[k])
        s[k] = v
    compare(s, run(s, "f32"), "f32")


@pytest.mark.parametrize("M", [2, 20, 130])
def test_scales_at_the_ends(M):
    """Zero, NaN and infinite scales reach their own rows and columns only."""
    s = make(4, M, 72, 64, "f32", bias=False)
    s["sx"][0], s["sw"][5], s["sw"][6] = 0.0, float("nan"), 0.0
    s["sx"][1] = float("nan")
    got = host(run(s, "f32"))
    assert np.isnan(got[1]).all() and np.isnan(got[:, 5]).all()
    keep = [c for c in range(72) if c != 5]
    assert not got[0, keep].any()
    rows = [r for r in range(M) if r != 1]
    if len(rows) > 1:
        y, sums, mag = oracle({**s, "sw": torch.nan_to_num(s["sw"]), "sx": torch.nan_to_num(s["sx"])})
        so.check(got[np.ix_(rows, keep)], y[np.ix_(rows, keep)], mag[np.ix_(rows, keep)], 8, "f32", "others")


def test_largest_k():
    """K at its limit with every product at its largest: the integer sum stays
    in range."""
    M, N, K = 3, 4, 65536
    s = make(5, M, N, K, "f32", bias=False)
    s["x"].fill_(-128), s["w"].fill_(-128)
    compare(s, run(s, "f32"), "f32")
    M = 24
    s = make(6, M, N, K, "f32", bias=False)
    s["x"].fill_(-128), s["w"].fill_(127)
    compare(s, run(s, "f32"), "f32")


def test_no_rows():
    gc.gconv_matmul_q8(16, 16, 16, 16, None, 16, gc.make_matmul_q8_problem(0, 8, 8), code("f32"), None)


def test_deterministic_and_on_another_stream():
    for M in (6, 60, 600):
        s = make(7, M, 520, 512, "bf16")
        a = run(s, "bf16")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            b = run(s, "bf16")
        assert same_bits(a, b)


@pytest.mark.parametrize("M", [4, 48, 300])
def test_graph_replay(M):
    s, other = make(8, M, 256, 192, "f32"), make(9, M, 256, 192, "f32")
    y = torch.empty(M, 256, device=DEV)
    p = gc.make_matmul_q8_problem(M, 256, 192)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gc.gconv_matmul_q8(s["x"], s["sx"], s["w"], s["sw"], s["b"], y, p, code("f32"), torch.cuda.current_stream())
    for k in s:
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    compare(other, y, "f32")


def test_output_past_32_bits():
    """Rows of y that start more than 2^31 elements in."""
    M, N, K = 3, 64, 64
    s = make(10, M, N, K, "bf16")
    stride = (1 << 30) + 64
    buf = torch.empty(2 * stride + N, dtype=torch.bfloat16, device=DEV)
    y = buf.as_strided((M, N), (stride, 1))
    gc.gconv_matmul_q8(s["x"], s["sx"], s["w"], s["sw"], s["b"], y, gc.make_matmul_q8_problem(M, N, K, stride), code("bf16"),
                       torch.cuda.current_stream())
    torch.cuda.synchronize()
    compare(s, y, "bf16")


# K shared by 2 ... 8 blocks: equal and ragged parts, rows and columns at their ends
SHARED = [(16, 128, 4096), (9, 130, 1040), (33, 65, 2000), (100, 1000, 3136), (300, 700, 4096), (16, 9000, 2048), (64, 5120, 4096),
          (150, 4000, 4112), (128, 1300, 8192)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHARED)
def test_shared_tiles(dtype, M, N, K):
    s = make(M + N + K, M, N, K, dtype)
    if dtype == "f16":
        s["sw"] /= 64  # keep sums inside the type's range
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("stride,offset", [(136, 4), (139, 0), (136, 1)])
def test_shared_tiles_into_strides(dtype, stride, offset):
    """Rows of y that take four values at a time, and rows that do not."""
    s = make(5, 20, 132, 1024, dtype, bias=False)
    compare(s, run(s, dtype, stride, offset), dtype)


def test_shared_tiles_are_exact_and_deterministic():
    s = make(6, 40, 300, 4096, "f32", top=7, bias=False)
    s["sx"].fill_(1.0), s["sw"].fill_(1.0)
    got = run(s, "f32")
    assert np.array_equal(host(got), oracle(s)[0])
    s = make(6, 40, 300, 4096, "f32")
    first = run(s, "f32")
    assert all(same_bits(run(s, "f32"), first) for _ in range(3))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M", range(1, 9))
@pytest.mark.parametrize("N,K", [(5, 2048), (1031, 2064), (130, 4096)])
def test_few_rows_with_a_long_sum(dtype, M, N, K):
    """Rows of one to eight tokens whose sums are shared by several warps."""
    s = make(M + N + K, M, N, K, dtype)
    if dtype == "f16":
        s["sw"] /= 64  # keep sums inside the type's range
    compare(s, run(s, dtype, N + 3 if M % 2 else 0), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 1001), (7, 129, 2050), (40, 700, 4099), (129, 131, 63), (65, 64, 65), (300, 1000, 777),
                                   (2100, 3001, 130), (1290, 4000, 197)])
def test_rows_of_any_width(dtype, M, N, K):
    """Widths that leave rows at every address, alone in a tile, sharing it, and
    several tiles a block."""
    s = make(M + N + K, M, N, K, dtype)
    if dtype == "f16":
        s["sw"] /= 64  # keep sums inside the type's range
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("shift", [1, 2, 3, 12])
@pytest.mark.parametrize("M,N,K", [(33, 140, 640), (260, 300, 1283)])
def test_rows_at_any_address(shift, M, N, K):
    s = make(7, M, N, K, "bf16")
    for k, at in (("x", shift), ("w", 5 - shift % 4)):
        buf = torch.empty(s[k].numel() + at, dtype=torch.int8, device=DEV)
        v = buf[at:].view(s[k].shape)
        v.copy_(s[k])
        s[k] = v
    compare(s, run(s, "bf16"), "bf16")


def test_two_threads_with_plans_of_different_sizes():
    """Calls from two threads and streams, one with tiles that need most of a block's
    shared memory, one with few: neither takes the other's away."""
    import threading

    cases = [(make(41, 600, 600, 256, "bf16"), 0), (make(42, 40, 130, 131, "bf16"), 0), (make(43, 33, 200, 48, "bf16"), 0),
             (make(44, 16, 128, 4096, "bf16"), 0)]
    want = [run(s, "bf16") for s, _ in cases]
    got, errors = [[] for _ in cases], []
    gate = threading.Barrier(len(cases))

    def work(k):
        s = cases[k][0]
        (M, K), N = s["x"].shape, s["w"].shape[0]
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            p, y = gc.make_matmul_q8_problem(M, N, K), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
            gate.wait(30)
            for _ in range(3000):
                gc.gconv_matmul_q8(s["x"], s["sx"], s["w"], s["sw"], s["b"], y, p, code("bf16"), st)
            st.synchronize()
            got[k].append(y)
        except Exception as e:  # noqa: BLE001
            errors.append(f"{(M, N, K)}: {e}")

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert same_bits(g[0], w)


@pytest.mark.parametrize("M,N,K", [(3, 5, 65536), (24, 40, 65536), (24, 40, 65531), (7, 130, 8192), (128, 1300, 8192), (2100, 3000, 4096),
                                   (1, 300, 4099), (40, 700, 4099), (300, 1000, 8191), (2100, 3000, 2053), (1290, 4000, 197)])
@pytest.mark.parametrize("shift", [0, 3])
def test_every_product_counts(M, N, K, shift):
    """Values up to 15 with fp32 outputs and scales of 1: sums stay below 2^24 for
    any K, so a single product lost or taken twice shows.  Rows of few and of many,
    shared tiles and whole ones, any width and address."""
    s = make(14, M, N, K, "f32", top=15, bias=False)
    s["sx"].fill_(1.0), s["sw"].fill_(1.0)
    if shift:
        for k, at in (("x", shift), ("w", 1)):
            buf = torch.empty(s[k].numel() + at, dtype=torch.int8, device=DEV)
            v = buf[at:].view(s[k].shape)
            v.copy_(s[k])
            s[k] = v
    want = s["x"].double() @ s["w"].double().t()  # exact: integers below 2^53
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(run(s, "f32").double(), want)
    s["x"].fill_(15), s["w"].fill_(15)  # and no two mistakes that cancel
    assert bool((run(s, "f32") == 225.0 * K).all())
