"""Forms of the selective scan that alignment, types and numbers of states choose, against the 64-bit walk: rows off
the vectors with every number of lanes, 16-bit types without a split, and bounds without a split's allowance."""
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
import ssm_oracle as so
from gpu_util import require_gpu
from seq_util import DEV, host, place
from test_gpu_ssm_scan import backward, check, forward, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def whole(d, G, lens=None):
    """The oracle with the bounds of a walk that is not split."""
    h = {k: host(v) for k, v in d.items()}
    return so.scan(h["x"], h["delta"], h["A"], h["Bm"], h["Cm"], h["skip"], h["z"], h["bias"], h["h0"],
                   None if lens is None else lens.tolist(), h.get("dy"), h.get("dhT"), G, parts=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,D,N,G", [(2, 1, 40, 16, 1), (2, 4, 33, 24, 1), (2, 40, 64, 8, 1), (1, 100, 64, 16, 1), (2, 70, 33, 5, 1),
                                       (2, 50, 35, 24, 1), (1, 33, 17, 32, 1), (2, 37, 9, 40, 1), (1, 60, 21, 64, 1), (1, 49, 66, 33, 3)])
def test_walks_without_a_split(B, T, D, N, G, dtype):
    d = tensors(B, T, D, N, G, dtype, train=True)
    p = gc.make_ssm_problem(B, T, D, N, G)
    assert gc.gconv_selective_scan_fwd_workspace_size(p, gc.DTYPE_CODES[dtype]) == 0
    y, hT, saved = forward(d, dtype, p, save=True)
    check({"y": y, "hT": hT, **backward(d, dtype, p, saved)}, whole(d, G), dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [7, 16, 21, 32, 64])
def test_odd_offsets_strides_and_lengths(N, dtype):
    """Column slices at odd elements of wider tensors (whose other elements are NaN), so that rows begin and end in the
    middle of a word; sequences of unlike lengths."""
    B, T, D = 3, 35, 26
    d = tensors(B, T, D, N, 1, dtype, train=True)
    wide, mixed, tm = (T * (2 * D + 3), 2 * D + 3), (T * (2 * N + 3), 2 * N + 3), (D + 1, B * (D + 1))
    e = {**d, "x": place(d["x"], (*wide, 1), 1), "z": place(d["z"], (*wide, 1), D + 2), "delta": place(d["delta"], (*wide, 1), 3),
         "Bm": place(d["Bm"], (*mixed, 1), 1), "Cm": place(d["Cm"], (*mixed, 1), N + 2), "dy": place(d["dy"], (*tm, 1), 1)}
    p = gc.make_ssm_problem(B, T, D, N, 1, x_stride=wide, z_stride=wide, delta_stride=wide, b_stride=mixed, c_stride=mixed, y_stride=tm)
    lens = torch.tensor([T, 17, 1], dtype=torch.int32, device=DEV)
    y, hT, saved = forward(e, dtype, p, lens=lens, save=True, y_stride=(*tm, 1))
    check({"y": y, "hT": hT, **backward(e, dtype, p, saved, lens=lens)}, whole(d, 1, lens), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,N,G", [(2, 3, 10, 16, 10), (2, 40, 10, 16, 10), (1, 20, 1, 1, 1), (3, 33, 14, 5, 7)])
def test_groups_of_few_channels(B, T, D, N, G, dtype):
    """A group of one channel, of two, and one channel alone."""
    d = tensors(B, T, D, N, G, dtype, train=True)
    p = gc.make_ssm_problem(B, T, D, N, G)
    y, hT, saved = forward(d, dtype, p, save=True)
    check({"y": y, "hT": hT, **backward(d, dtype, p, saved)}, whole(d, G), dtype)
