"""The 8-bit floating-point product at sizes that go to pairs of blocks (f8_pairs.py): every type, format, kind of
scale and alignment against 64 bits, and beside other calls."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import f8_pairs as fp
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, host, same_bits
from test_gpu_f8_matmul import DT, check, operand, product, reference
from test_gpu_ssm_calls import Norm, Product, Scan, alone, empty, expect, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("M,N,K", fp.PAIRS)
@pytest.mark.parametrize("dtype,xf,wf,w_rows,bias", [("f32", "e4m3", "e4m3", 128, True), ("f16", "e4m3", "e4m3", 128, False),
                                                     ("bf16", "e5m2", "e4m3", 128, False), ("bf16", "e4m3", "e5m2", 1, True),
                                                     ("f16", "e5m2", "e5m2", 1, False), ("f32", "e5m2", "e4m3", 1, False)])
def test_against_64_bits(M, N, K, dtype, xf, wf, w_rows, bias):
    x, sx = operand(M, K, xf, M, 1)
    w, sw = operand(N, K, wf, -(-N // w_rows), 2)
    # e5m2's values here reach 57344, e4m3's 448: sums within f16's range
    sx *= 2.0 ** -(6 + 6 * ((xf == "e5m2") + (wf == "e5m2"))) if dtype == "f16" else 1.0
    b = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(DT[dtype]).to(DEV) if bias else None
    y = product(x, sx, w, sw, b, M, N, K, dtype, xf, wf, w_rows)
    check(y, *reference(x, sx, w, sw, b, M, N, K, xf, wf, w_rows), dtype)


@pytest.mark.parametrize("w_rows", [1, 128])
def test_exact_where_every_sum_is_whole(w_rows):
    """Small integers and powers of two for scales: to the bit."""
    M, N, K = fp.EXACT
    x, sx = operand(M, K, "e4m3", M, 5, integers=True)
    w, sw = operand(N, K, "e4m3", -(-N // w_rows), 6, integers=True)
    y = product(x, sx, w, sw, None, M, N, K, "f32", w_rows=w_rows)
    ref, _ = reference(x, sx, w, sw, None, M, N, K, "e4m3", "e4m3", w_rows)
    assert np.array_equal(host(y), ref)


@pytest.mark.parametrize("dtype,y_stride", [("bf16", 2104), ("bf16", 2107), ("f32", 2102), ("f16", 2103)])
def test_pitches_and_strides(dtype, y_stride):
    """Wider rows and scales of a longer matrix with NaN in between; rows of y with a stride, on and off 16 bytes."""
    M, N, K = fp.STRIDED
    x, sx = operand(M, K, "e4m3", M + 9, 1, pitch=544)
    w, sw = operand(N, K, "e4m3", N + 3, 2, pitch=528)
    sx *= 2.0 ** -6
    p = gc.make_matmul_f8_problem(M, N, K, 0, 0, 1, x_pitch=544, x_scale_stride=M + 9, w_pitch=528, w_scale_stride=N + 3, y_stride=y_stride)
    y = Guarded((M, N), DT[dtype], (y_stride, 1))
    gc.gconv_matmul_f8(x, sx, w, sw, None, y.t, p, code(dtype), torch.cuda.current_stream())
    ref, lim = reference(x, sx[:, :M], w, sw[:, :N], None, M, N, K, "e4m3", "e4m3", 1)
    check(y.check(), ref, lim, dtype)


@pytest.mark.parametrize("w_rows", [1, 128])
def test_not_finite_values_reach_their_rows_and_columns_only(w_rows):
    """In rows of both blocks of a pair, and in a row of wq."""
    M, N, K = fp.STRIDED
    x, sx = operand(M, K, "e4m3", M, 1)
    w, sw = operand(N, K, "e4m3", -(-N // w_rows), 2)
    clean = product(x, sx, w, sw, None, M, N, K, "bf16", w_rows=w_rows)
    x[3, 5] = x[130, 519] = w[2099, 0] = 0x7F  # NaN
    sx[4, 1099] = float("nan")
    y = product(x, sx, w, sw, None, M, N, K, "bf16", w_rows=w_rows)
    rows = [k for k in range(M) if k not in (3, 130, 1099)]
    assert bool(y[[3, 130, 1099]].isnan().all()) and bool(y[:, 2099].isnan().all())
    assert same_bits(y[rows, :2099], clean[rows, :2099])


def work(seed):
    """Pairs of one and of two rounds, with scales of both kinds, among other kernels."""
    one, two, even, _ = fp.CALLS
    return [Product(*one, 128, seed), Scan(1, 300, 64, 16, "bf16", seed + 1), Product(*two, 1, seed + 2),
            Product(*fp.OTHERS[0], 128, seed + 3), Norm(40, 2048, "bf16", seed + 4), Product(*even, 128, seed + 5)]


def test_one_after_the_other():
    """Without a pause: blocks of a call begin where the pairs of the one before end."""
    jobs = work(1)
    want = alone(jobs)
    for _ in range(20):
        for j in jobs + jobs[::-1]:
            j.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    expect(jobs, want)


def test_two_streams_and_two_graphs_at_once():
    jobs, streams, graphs = [work(20), work(40)], [torch.cuda.Stream(), torch.cuda.Stream()], []
    want = [alone(j) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, b in zip(jobs[0], jobs[1][::-1]):
            a.run(streams[0])
            b.run(streams[1])
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        expect(j, w)
    for j, stream in zip(jobs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for job in j:
                job.run(stream)
        graphs.append(graph)
    for j in jobs:
        for job in j:
            job.x.mul_(-0.5)
    want = [alone(j) for j in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        expect(j, w)


def test_beside_the_products_of_8_bit_integers():
    """Tensor memory passes between the two kinds, in one stream and across two."""
    M, N, K = fp.CALLS[3]
    f8 = Product(M, N, K, 128, 100)
    g = torch.Generator().manual_seed(101)
    xq, wq = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).to(DEV) for n in (M, N))
    sx, sw, y = randn(g, M).abs(), randn(g, N).abs(), empty(M, N, dtype=torch.bfloat16)
    p = gc.make_matmul_q8_problem(M, N, K)

    def q8(stream):
        gc.gconv_matmul_q8(xq, sx, wq, sw, None, y, p, code("bf16"), stream)
    want = alone([f8])
    q8(torch.cuda.current_stream())
    torch.cuda.synchronize()
    y_want = y.clone()
    y.zero_()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(20):
        f8.run(torch.cuda.current_stream())
        q8(torch.cuda.current_stream() if k % 2 else other)
        f8.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    expect([f8], want)
    assert same_bits(y, y_want)
