"""The gated scan where its gates and rates come to their ends, against 64 bits
within bounds followed channel by channel (seq_bounds.py)."""
import numpy as np
import pytest
import torch

import seq_bounds as sb
from gpu_util import require_gpu
from seq_util import DEV, f64, host, randn
from test_gpu_seq_scan import C, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def compare(s, got, dtype, backward=True):
    x, r, i, lam, h0, dy, dhT = f64(*(s[k] for k in ("x", "r", "i", "lam", "h0", "dy", "dhT")))
    lens = None if s["lens"] is None else s["lens"].cpu().numpy()
    if lens is not None:
        x, r, i, dy = (np.nan_to_num(v) for v in (x, r, i, dy))
    want = sb.forward(x, r, i, lam, h0, lens, C)
    if backward:
        want.update(sb.backward(dy, dhT, x, r, i, lam, h0, lens, C))
    for k in ("y", "hT", "dx", "dr", "di", "dlam", "dh0"):
        if k in want:
            sb.check(host(got[k]), *want[k], "f32" if k in ("hT", "dlam", "dh0") else dtype, k)


ODD = {k: (150 * 69 + 3, 69) for k in ("x", "r", "i", "y")}  # rows that TMA cannot take


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,lens,strides", [(1, None, None), (2, None, None), (37, None, None), (64, None, None),
                                            (150, [150, 0, 1, 70], None), (150, [3, 149, 16, 8], ODD), (150, None, ODD)])
def test_infinite_rates(dtype, T, lens, strides):
    """lam of infinity, and rates that pass fp32: a = 0 and s = 1, the formulas'
    limits, also where a tile reaches past the sequence's end; the gradients of r
    and lam are 0."""
    s = make(21, 4, T, 64, dtype, lens)
    s["lam"][3], s["lam"][10:12], s["lam"][40] = float("inf"), 3e38, 1e20
    got = run(s, dtype, strides)
    compare(s, got, dtype)
    for k in ("dr", "dlam"):
        assert not got[k][..., [3, 10, 11, 40]].any(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_lost_rate_stays_in_its_channel(dtype):
    s = make(22, 2, 70, 64, dtype)
    s["lam"][6] = float("nan")
    got = run(s, dtype)
    assert bool(torch.isnan(got["y"][..., 6]).all()) and bool(torch.isnan(got["hT"][..., 6]).all())
    keep = [k for k in range(64) if k != 6]
    sub = {k: v if v is None else v[..., keep] for k, v in s.items()}
    compare({**sub, "lens": None}, {k: v[..., keep] for k, v in got.items()}, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D,strides", [(2, 64, None), (96, 64, None), (150, 64, ODD), (61, 95, None)])
@pytest.mark.parametrize("kind", ["slow", "wide", "fast"])
def test_open_and_shut_gates(dtype, T, D, strides, kind):
    """Gates from -30 to 30: the gradients of open ones hold 1 - sig, which must not
    be a difference from 1."""
    s = make(23, 2, T, D, dtype, lam="slow" if kind == "slow" else "wide")
    if kind == "fast":
        s["lam"] = s["lam"] + 12
    g = torch.Generator().manual_seed(24)
    for k in ("r", "i"):
        s[k] = (torch.rand(2, T, D, generator=g) * 60 - 30).to(DEV).to(s["x"].dtype)
    compare(s, run(s, dtype, strides), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [8.0, 12.0, 16.0, 17.0, 20.0, 30.0, 60.0])
def test_gradients_of_open_gates(dtype, gate):
    """One value for every gate: a gradient that vanished or changed its sign would
    do so everywhere."""
    s = make(25, 1, 40, 64, dtype)
    s["r"].fill_(gate), s["i"].fill_(gate)
    got = run(s, dtype)
    compare(s, got, dtype)
    assert bool((got["di"] != 0).all()) and bool((got["dr"] != 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,strides", [(1, None), (40, None), (150, ODD)])
@pytest.mark.parametrize("top", [50.0, 1e4, 1e15, 1e29])
def test_steep_channels_with_shut_gates(dtype, T, strides, top):
    """A steep channel's factor is far from 0 where its gate is shut as far as
    exp(-88): one token or many, it is there."""
    s = make(26, 2, T, 64, dtype)
    g = torch.Generator().manual_seed(27)
    s["lam"] = (torch.rand(64, generator=g) * top + 6).to(DEV)
    s["r"] = (torch.rand(2, T, 64, generator=g) * 12 - 94).to(DEV).to(s["x"].dtype)
    s["h0"].zero_()
    got = run(s, dtype)
    compare(s, got, dtype, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 192), (100, 192), (61, 95)])
def test_each_channel_by_its_own_rate(dtype, T, D):
    """Slow, plain, still and steep channels beside each other, each within the
    bound of its own rate."""
    s = make(28, 2, T, D, dtype)
    u = torch.rand(D, generator=torch.Generator().manual_seed(29)).to(DEV)
    kind = torch.arange(D, device=DEV) // 32 % 6
    lam = torch.where(kind == 1, u * 4 - 3.3, s["lam"])
    lam = torch.where((kind == 2) | (kind == 3), u - 30, lam)
    s["lam"] = torch.where(kind == 5, u + 5, lam)
    compare(s, run(s, dtype), dtype)


@pytest.mark.parametrize("dtype,T", [("f32", 6000), ("bf16", 20000)])
def test_the_state_of_a_long_sequence(dtype, T):
    """The carried state keeps fp32: its bound forgets as the channel does."""
    s = make(30, 1, T, 64, dtype)
    compare(s, run(s, dtype, backward=False), dtype, backward=False)


def test_the_gradients_of_a_long_sequence():
    s = make(31, 1, 5000, 64, "f32", [4990])
    compare(s, run(s, "f32"), "f32")
