"""The selective scan's decays over the whole range of their arguments: growing states in a walk that is split, and
states that decay by a little over thousands of tokens."""
import numpy as np
import pytest
import torch

import depthwise_convolution_forward_gb300 as gc
from gpu_util import require_gpu
from seq_util import DEV, code
from test_gpu_ssm_scan import check, forward, oracle, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def growing(T, D, N):
    """Positive A, steps near 0.7: a part of 64 tokens multiplies its first state by up to exp(130), more than fp32
    holds, and the state is 0 until the last tokens.  The gradients are 0 but for the first ones."""
    d = tensors(1, T, D, N, 1, "f32", train=True, gate=False)
    g = torch.Generator().manual_seed(T + D)
    d["A"] = (torch.rand(D, N, generator=g) + 2).to(DEV)
    d["delta"], d["bias"] = d["delta"] * 0.1, None
    d["h0"], d["dhT"] = None, None
    d["x"][:, :-8] = 0
    d["dy"][:, 8:] = 0
    return d


@pytest.mark.parametrize("T,D,N", [(1024, 64, 16), (700, 33, 5)])
def test_growing_states_in_parts(T, D, N):
    d = growing(T, D, N)
    p = gc.make_ssm_problem(1, T, D, N)
    assert gc.gconv_selective_scan_fwd_workspace_size(p, code("f32")) > 0  # a split walk
    out = {}
    saved = torch.zeros(gc.gconv_selective_scan_saved_size(p, code("f32")), dtype=torch.uint8, device=DEV)
    ws = torch.zeros(gc.gconv_selective_scan_fwd_workspace_size(p, code("f32")), dtype=torch.uint8, device=DEV)
    wb = torch.zeros(gc.gconv_selective_scan_bwd_workspace_size(p, code("f32")), dtype=torch.uint8, device=DEV)
    y, hT = torch.empty_like(d["x"]), torch.empty(1, D, N, device=DEV)
    gc.gconv_selective_scan_fwd(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["skip"], None, None, None, None, y, hT, saved, p,
                                code("f32"), ws, 0, torch.cuda.current_stream())
    like = {"dx": "x", "ddelta": "delta", "dA": "A", "dBm": "Bm", "dCm": "Cm", "dskip": "skip"}
    out = {k: torch.empty_like(d[v]) for k, v in like.items()}
    gc.gconv_selective_scan_bwd(d["dy"], None, d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["skip"], None, None, None, saved,
                                out["dx"], out["ddelta"], out["dA"], out["dBm"], out["dCm"], out["dskip"], None, None, None, p,
                                code("f32"), wb, 0, torch.cuda.current_stream())
    ref = oracle(d, 1)
    assert all(np.isfinite(ref[k][0]).all() for k in ("y", "hT", *out))
    check({"y": y, "hT": hT, **out}, ref, "f32")


def test_a_tiny_state_grows_by_more_than_fp32_holds():
    """h0 = 1e-30, and one part's tokens multiply it by exp(102) = 2.9e44."""
    T, D, N = 1024, 64, 4
    d = tensors(1, T, D, N, 1, "f32", gate=False)
    for k in ("x", "delta"):
        d[k].zero_()
    d["delta"][:, 128:192] = 1.0
    d["A"], d["bias"], d["h0"] = torch.full((D, N), 1.6, device=DEV), None, torch.full((1, D, N), 1e-30, device=DEV)
    p = gc.make_ssm_problem(1, T, D, N, softplus=False)
    y, hT, _ = forward(d, "f32", p)
    check({"y": y, "hT": hT}, oracle(d, 1, soft=False), "f32")


@pytest.mark.parametrize("B,T,D,N,calls", [(2, 2048, 9728, 4, 1), (1, 4096, 64, 16, 1), (64, 4, 64, 16, 512)])
def test_slow_decays_lean_to_no_side(B, T, D, N, calls):
    """States that lose 1e-4 to 3e-3 of themselves in base 2 a token, in a whole walk, in parts and by few tokens: the
    mean error of a token's decay, over all states, is below 2^-27 (an eighth of a rounding's half step).  Roundings
    themselves, 2^-24 at most and of either sign, leave 2^-24 / sqrt(4e6) in the mean of 4e6 or more tokens and states."""
    g = torch.Generator(device=DEV).manual_seed(T)
    A = -(1 + torch.rand(D, N, generator=g, device=DEV)) * 0.6931
    zero, mix = torch.zeros(B, T, D, device=DEV), torch.zeros(B, T, N, device=DEV)
    h, total, y = torch.ones(B, D, N, device=DEV), 0.0, torch.empty(B, T, D, device=DEV)
    p = gc.make_ssm_problem(B, T, D, N, softplus=False)
    need = gc.gconv_selective_scan_fwd_workspace_size(p, code("f32"))
    assert (need > 0) == (T == 4096)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    for _ in range(calls):
        delta = 1e-4 * torch.exp(torch.rand(B, T, D, generator=g, device=DEV) * float(np.log(15)))
        gc.gconv_selective_scan_fwd(zero, delta, A, mix, mix, None, None, None, h, None, y, h, None, p, code("f32"), ws, 0,
                                    torch.cuda.current_stream())
        total = total + delta.double().sum(1)
    lost = torch.log(h.double()) - total[..., None] * A.double()
    mean = float(lost.mean()) / (T * calls)
    assert abs(mean) < 2.0 ** -27, mean


@pytest.mark.parametrize("T", [4, 40, 2100])
def test_states_that_never_decay_beside_fast_ones(T):
    """A of 0 beside A of -1 to -3 among a channel's states: to the bit what comes in, in every form of the walk."""
    B, D, N = 2, 70, 12
    d = tensors(B, T, D, N, 1, "f32", gate=False)
    d["A"][:, ::3], d["x"] = 0.0, torch.zeros_like(d["x"])
    y, hT, _ = forward(d, "f32", gc.make_ssm_problem(B, T, D, N))
    assert torch.equal(hT[..., ::3], d["h0"][..., ::3])
