"""The norm to 8-bit floating point with its residual written in the place of an input, at widths and strides of each
form: the same bits as out of place."""
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
from gpu_util import require_gpu
from seq_util import DEV, Guarded, code, place, same_bits
from test_gpu_f8_quant import DT, f8_out, matrix, norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,D,stride", [(5, 136, 136), (900, 101, 101), (900, 1001, 1003), (40, 4095, 4095), (3, 20001, 20001)])
@pytest.mark.parametrize("where", ["x", "residual"])
def test_in_place(M, D, stride, dtype, where):
    x, res = matrix(M, D, dtype, 1, 1.0), matrix(M, D, dtype, 2, 1.0)
    want = norm(x, res, None, dtype)
    wx, wr = Guarded((M, D), DT[dtype], (stride, 1), 1), Guarded((M, D), DT[dtype], (stride, 1), 1)
    wx.t.copy_(x)
    wr.t.copy_(res)
    out = wx.t if where == "x" else wr.t
    y, (q, s) = Guarded((M, D), DT[dtype]), f8_out(M, D)
    gc.gconv_rms_norm_f8(wx.t, wr.t, None, out, y.t, q.t, s.t, gc.GCONV_E4M3, gc.make_norm_problem(M, D, 1e-6, stride, stride), code(dtype),
                         torch.cuda.current_stream())
    got = [wx.check() if where == "x" else wr.check(), y.check(), q.check(), s.check()]
    assert all(same_bits(a, b) for a, b in zip(got, want))
    assert same_bits(wr.t if where == "x" else wx.t, res if where == "x" else x)


def test_in_place_without_a_residual():
    x = matrix(300, 333, "bf16", 4)
    p = gc.make_norm_problem(300, 333, 1e-6)
    out, was = place(x, (333, 1)), x.clone()
    y = torch.empty_like(x)
    gc.gconv_rms_norm_f8(out, None, None, out, y, None, None, gc.GCONV_E4M3, p, code("bf16"), torch.cuda.current_stream())
    assert same_bits(out, was) and same_bits(y, norm(x, None, None, "bf16", want_q=False)[1])
    assert out.device == DEV
