"""Host-side checks of the sequence operators' C ABI: exported symbols, record
layouts, refusals before any launch.  No GPU needed."""
import ctypes
import os
import re
import subprocess

import pytest

import depthwise_convolution_forward_gb300 as gc
from depthwise_convolution_forward_gb300 import _binding as B
from depthwise_convolution_forward_gb300 import _seq, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = B.GCONV_F32, B.GCONV_BF16
INVALID, UNSUPPORTED = B.GCONV_ERR_INVALID_ARG, B.GCONV_ERR_UNSUPPORTED
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.load_library()


def refused(status, fn, *args, says=None):
    with pytest.raises(gc.GconvError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)
    if says:
        assert says in gc.gconv_last_error()


def test_header_symbols_exported(lib):
    src = open(os.path.join(ROOT, "include", "gconv_seq.h")).read()
    consts = dict(re.findall(r"#define (GCONV_[A-Z0-9_]+) ([0-9]+)\s*$", src, flags=re.M))
    assert int(consts["GCONV_SCAN_CHUNK"]) == _seq.GCONV_SCAN_CHUNK
    assert int(consts["GCONV_CONV1D_MAX_K"]) == _seq.GCONV_CONV1D_MAX_K
    assert int(consts["GCONV_NORM_MAX_D"]) == _seq.GCONV_NORM_MAX_D
    assert int(consts["GCONV_MATMUL_Q8_MAX_K"]) == _seq.GCONV_MATMUL_Q8_MAX_K
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^\s*gconv_status\s+([a-z_0-9]+)\s*\(", src, flags=re.M)))
    assert len(names) == 10, names
    out = subprocess.run(["nm", "-D", "--defined-only", B.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    for n in names:
        assert n in exported and hasattr(gc, n), n


def test_record_layouts():
    assert ctypes.sizeof(gc.gconv_conv1d_problem) == 64 and gc.gconv_conv1d_problem.x_stride.offset == 32
    assert ctypes.sizeof(gc.gconv_scan_problem) == 88 and gc.gconv_scan_problem.x_stride.offset == 24
    assert ctypes.sizeof(gc.gconv_norm_problem) == 48 and gc.gconv_norm_problem.x_stride.offset == 16
    assert ctypes.sizeof(gc.gconv_matmul_q8_problem) == 32 and gc.gconv_matmul_q8_problem.y_stride.offset == 16


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "gconv_seq.h"\nint main(void) { gconv_scan_problem p = {1, 1, 1, 8.0f}; return sizeof(p) != 88; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o",
                    str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")]).returncode == 0


# distinct, far-apart made-up device addresses: a refusal touches none of them
A = [(k + 1) * 64 * MB for k in range(20)]


def scan_fwd(p, dt=F32, x=A[0], r=A[1], i=A[2], lam=A[3], h0=A[4], lens=None, y=A[5], hT=A[6], saved=None):
    gc.gconv_gated_scan_fwd(x, r, i, lam, h0, lens, y, hT, saved, p, dt, None)


def scan_bwd(p, dt=F32, ws=A[12], n=1 << 40, **kw):
    a = dict(dy=A[0], dhT=A[1], x=A[2], r=A[3], i=A[4], lam=A[5], lens=None, saved=A[6], dx=A[7], dr=A[8], di=A[9],
             dlam=A[10], dh0=A[11])
    a.update(kw)
    gc.gconv_gated_scan_bwd(*a.values(), p, dt, ws, n, None)


GOOD_SCAN = dict(b=2, t=10, d=64)


@pytest.mark.parametrize("bad", [dict(b=0), dict(t=0), dict(d=0), dict(b=-1), dict(decay=0.0), dict(decay=-1.0),
                                 dict(decay=float("inf")), dict(decay=float("nan")), dict(x_stride=(640, 63)),
                                 dict(r_stride=(600, 64)), dict(i_stride=(-640, 64)), dict(y_stride=(640, -64)),
                                 dict(x_stride=(0, 64)), dict(y_stride=(1 << 62, 64)), dict(b=1 << 41),
                                 dict(b=1 << 20, d=1 << 20)])
def test_scan_problem_refused(bad):
    p = gc.make_scan_problem(**{**GOOD_SCAN, **bad})
    refused(INVALID, scan_fwd, p)
    refused(INVALID, scan_bwd, p)
    refused(INVALID, gc.gconv_gated_scan_saved_size, p, F32)
    refused(INVALID, gc.gconv_gated_scan_bwd_workspace_size, p, F32)


def test_scan_arguments_refused():
    p = gc.make_scan_problem(**GOOD_SCAN)
    refused(UNSUPPORTED, scan_fwd, p, 7)
    refused(UNSUPPORTED, gc.gconv_gated_scan_saved_size, p, 9)
    for k in ("x", "r", "i", "lam", "y"):
        with pytest.raises(gc.GconvError) as e:
            scan_fwd(p, **{k: None})
        assert e.value.status == INVALID
    for k in ("dy", "x", "r", "i", "lam", "saved", "dx", "dr", "di", "dlam"):
        with pytest.raises(gc.GconvError) as e:
            scan_bwd(p, **{k: None})
        assert e.value.status == INVALID
    for kw in (dict(y=A[0]), dict(y=A[1] + 64), dict(y=A[4]), dict(hT=A[4] + 4), dict(hT=A[5]), dict(hT=A[3]),
               dict(saved=A[5]), dict(saved=A[4]), dict(lens=A[6])):
        with pytest.raises(gc.GconvError):
            scan_fwd(p, **kw)
        assert "overlaps" in gc.gconv_last_error()
    with pytest.raises(gc.GconvError):
        scan_fwd(p, saved=A[8] + 4)
    assert "aligned" in gc.gconv_last_error()
    for kw in (dict(dx=A[8]), dict(dr=A[2]), dict(di=A[0] + 4), dict(dlam=A[5]), dict(dh0=A[1]), dict(dlam=A[11]),
               dict(ws=A[7]), dict(saved=A[9])):
        with pytest.raises(gc.GconvError):
            scan_bwd(p, **kw)
        assert "overlaps" in gc.gconv_last_error()
    need = gc.gconv_gated_scan_bwd_workspace_size(p, F32)
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=A[12] + 8)):
        with pytest.raises(gc.GconvError):
            scan_bwd(p, **kw)
        assert "workspace" in gc.gconv_last_error()


def test_column_slices_are_told_from_overlaps():
    """x, r, i and their gradients as slices of one buffer pass the checks; slices
    that share a column do not."""
    st = (10 * 192, 192)
    p = gc.make_scan_problem(**GOOD_SCAN, x_stride=st, r_stride=st, i_stride=st)
    e = 4 * 64
    with pytest.raises(gc.GconvError):  # dr meets dx's last column
        scan_bwd(p, dx=A[7], dr=A[7] + e - 4, di=A[7] + 2 * e)
    assert "overlaps" in gc.gconv_last_error()
    with pytest.raises(gc.GconvError):  # di runs over the end of the pitch into dx
        scan_bwd(p, dx=A[7], dr=A[7] + e, di=A[7] + 2 * e + 4)
    assert "overlaps" in gc.gconv_last_error()
    with pytest.raises(gc.GconvError):  # fine slices: refused for its workspace alone
        scan_bwd(p, dx=A[7], dr=A[7] + e, di=A[7] + 2 * e, ws=None)
    assert "workspace" in gc.gconv_last_error()


def conv_fwd(p, dt=F32, x=A[0], w=A[1], bias=A[2], state_in=A[3], lens=None, y=A[4], state_out=A[5]):
    gc.gconv_causal_conv1d_fwd(x, w, bias, state_in, lens, y, state_out, p, dt, None)


def conv_bwd(p, dt=F32, ws=A[12], n=1 << 40, **kw):
    a = dict(dy=A[0], dso=A[1], x=A[2], w=A[3], bias=A[4], state_in=A[5], lens=None, dx=A[6], dw=A[7], dbias=A[8], dsi=A[9])
    a.update(kw)
    gc.gconv_causal_conv1d_bwd(*a.values(), p, dt, ws, n, None)


GOOD_CONV = dict(b=2, t=10, d=64, k=4)


@pytest.mark.parametrize("bad", [dict(b=0), dict(t=0), dict(d=0), dict(k=0), dict(k=9), dict(act=2), dict(act=-1),
                                 dict(x_stride=(640, 60)), dict(y_stride=(64, 64))])
def test_conv_problem_refused(bad):
    p = gc.make_conv1d_problem(**{**GOOD_CONV, **bad})
    refused(INVALID, conv_fwd, p)
    refused(INVALID, conv_bwd, p)
    refused(INVALID, gc.gconv_causal_conv1d_bwd_workspace_size, p, F32)


def test_conv_arguments_refused():
    p = gc.make_conv1d_problem(**GOOD_CONV)
    refused(UNSUPPORTED, conv_fwd, p, 3)
    q = gc.make_conv1d_problem(**GOOD_CONV)
    q.reserved = 1
    refused(INVALID, conv_fwd, q)
    for k in ("x", "w", "y"):
        with pytest.raises(gc.GconvError):
            conv_fwd(p, **{k: None})
    for k in ("dy", "x", "w", "dx", "dw"):
        with pytest.raises(gc.GconvError):
            conv_bwd(p, **{k: None})
    for kw in (dict(y=A[0]), dict(y=A[3]), dict(state_out=A[3] + 4), dict(state_out=A[4]), dict(state_out=A[1]),
               dict(lens=A[4]), dict(y=A[2] - 4)):
        with pytest.raises(gc.GconvError):
            conv_fwd(p, **kw)
        assert "overlaps" in gc.gconv_last_error()
    for kw in (dict(dx=A[2]), dict(dw=A[3]), dict(dbias=A[4]), dict(dsi=A[5]), dict(dsi=A[1]), dict(dx=A[0]), dict(ws=A[6])):
        with pytest.raises(gc.GconvError):
            conv_bwd(p, **kw)
        assert "overlaps" in gc.gconv_last_error()
    need = gc.gconv_causal_conv1d_bwd_workspace_size(p, F32)
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=A[12] + 4)):
        with pytest.raises(gc.GconvError):
            conv_bwd(p, **kw)
        assert "workspace" in gc.gconv_last_error()


def norm(p, dt=F32, x=A[0], res=A[1], w=A[2], ro=A[3], y=A[4], q=A[5], scale=A[6]):
    gc.gconv_rms_norm_q8(x, res, w, ro, y, q, scale, p, dt, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=32769), dict(eps=-1e-6),
                                 dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=63), dict(y_stride=-64),
                                 dict(residual_stride=1)])
def test_norm_problem_refused(bad):
    p = gc.make_norm_problem(**{**dict(rows=4, d=64), **bad})
    refused(INVALID, norm, p)
    refused(INVALID, gc.gconv_quantize_rows_q8, A[0], A[1], A[2], p, F32)


def test_norm_arguments_refused():
    p = gc.make_norm_problem(4, 64)
    refused(UNSUPPORTED, norm, p, 3)
    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(y=None, q=None, scale=None)):
        with pytest.raises(gc.GconvError) as e:
            norm(p, **kw)
        assert e.value.status == INVALID
    for kw in (dict(y=A[0]), dict(q=A[1]), dict(scale=A[2]), dict(ro=A[0] + 4), dict(ro=A[1] - 4), dict(ro=A[4]),
               dict(q=A[4]), dict(ro=A[2])):
        with pytest.raises(gc.GconvError):
            norm(p, **kw)
        assert "overlaps" in gc.gconv_last_error()
    for a in ((None, A[1], A[2]), (A[0], None, A[2]), (A[0], A[1], None), (A[0], A[0], A[2])):
        refused(INVALID, gc.gconv_quantize_rows_q8, *a, p, F32)


@pytest.mark.parametrize("bad", [dict(m=-1), dict(m=1 << 31), dict(n=0), dict(n=(1 << 21) + 1), dict(k=0), dict(k=65537),
                                 dict(y_stride=63), dict(y_stride=1 << 62)])
def test_matmul_problem_refused(bad):
    p = gc.make_matmul_q8_problem(**{**dict(m=4, n=64, k=64), **bad})
    refused(INVALID, gc.gconv_matmul_q8, A[0], A[1], A[2], A[3], A[4], A[5], p, F32)


def test_matmul_arguments_refused():
    p = gc.make_matmul_q8_problem(4, 64, 64)
    refused(UNSUPPORTED, gc.gconv_matmul_q8, A[0], A[1], A[2], A[3], A[4], A[5], p, 5)
    for k in (0, 1, 2, 3, 5):
        a = [A[0], A[1], A[2], A[3], A[4], A[5]]
        a[k] = None
        refused(INVALID, gc.gconv_matmul_q8, *a, p, F32)
    for k in range(5):
        refused(INVALID, gc.gconv_matmul_q8, A[0], A[1], A[2], A[3], A[4], A[k], p, BF16, says="overlaps")


def test_null_problem_refused(lib):
    for name, n in (("gconv_gated_scan_fwd", 9), ("gconv_causal_conv1d_fwd", 7), ("gconv_rms_norm_q8", 7),
                    ("gconv_quantize_rows_q8", 3), ("gconv_matmul_q8", 6)):
        assert getattr(lib, name)(*[None] * n, None, F32, None) == INVALID


def test_sizes_depend_on_the_problem_only():
    p = gc.make_scan_problem(3, 33, 70)
    assert gc.gconv_gated_scan_saved_size(p, F32) == 3 * -(-33 // _seq.GCONV_SCAN_CHUNK) * 70 * 4 == gc.gconv_gated_scan_saved_size(p, BF16)
    assert gc.gconv_gated_scan_bwd_workspace_size(p, F32) >= 70 * 4
    q = gc.make_conv1d_problem(3, 33, 70, 4)
    assert gc.gconv_causal_conv1d_bwd_workspace_size(q, F32) >= 70 * 5 * 4


@pytest.mark.parametrize("d", [(1 << 31) - 127, (1 << 31) - 1])
def test_widths_past_the_limit_are_refused(d):
    """The last channels that 32 bits count would overflow a launch's rounding up."""
    p = gc.make_scan_problem(1, 2, d)
    refused(INVALID, gc.gconv_gated_scan_saved_size, p, BF16, says="D must be")
    refused(INVALID, gc.gconv_gated_scan_bwd_workspace_size, p, BF16, says="D must be")
    refused(INVALID, scan_fwd, p, BF16, says="D must be")
    q = gc.make_conv1d_problem(1, 2, d, 4)
    refused(INVALID, gc.gconv_causal_conv1d_bwd_workspace_size, q, BF16, says="D must be")
    refused(INVALID, conv_fwd, q, BF16, says="D must be")


def test_the_widest_rows_are_taken():
    d = _seq.GCONV_SEQ_MAX_D
    assert d == (1 << 31) - 128
    assert gc.gconv_gated_scan_saved_size(gc.make_scan_problem(1, 2, d), BF16) == 4 * d
    assert gc.gconv_causal_conv1d_bwd_workspace_size(gc.make_conv1d_problem(1, 2, d, 4), BF16) == 20 * d
