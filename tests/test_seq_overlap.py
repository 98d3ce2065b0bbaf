"""Overlap checks of the sequence operators, on the CPU: the C ABI built with launches
that do nothing (``tests/harness/api_seq.cu``), its answers compared with the elements
that the tensors really share."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import depthwise_convolution_forward_gb300 as gc
from depthwise_convolution_forward_gb300 import _binding as B
from depthwise_convolution_forward_gb300 import _seq

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
OK, INVALID, F32 = 0, B.GCONV_ERR_INVALID_ARG, B.GCONV_F32
BASE, FAR = 1 << 30, 1 << 42  # made-up addresses


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    so = str(tmp_path_factory.mktemp("api") / "api_seq.so")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr", "-w", "-shared",
                    "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "harness", "api_seq.cu"), "-o",
                    so], check=True)
    lib = ctypes.CDLL(so)
    before = _seq._fn
    _seq.declare(lib)
    _seq._fn = before  # the package keeps calling its own library
    return lib


def conv(lib, p, x, y):
    """Status of a forward call on x and y at these addresses."""
    return lib.gconv_causal_conv1d_fwd(x, FAR, None, None, None, y, None, p, F32, None)


def elements(at, b, t, d, stride):
    return {at // 4 + i * stride[0] + j * stride[1] + k for i in range(b) for j in range(t) for k in range(d)}


def test_token_and_sequence_ranges_of_one_buffer(lib):
    """Two ranges of the tokens, or of the sequences, of one [B, T, D] buffer do not
    overlap, in batch-major and in time-major order; ranges that share a row do."""
    bm, tm = (20 * 64, 64), (64, 6 * 64)  # [., 20, 64]; [., 6, 64] with time outermost
    for st, b, t, step, n in ((bm, 3, 10, 64, 10), (tm, 2, 7, 64, 2), (tm, 6, 3, 6 * 64, 3), (bm, 2, 20, 20 * 64, 2)):
        p = gc.make_conv1d_problem(b, t, 64, 4, 0, st, st)
        for rows in range(-n, n + 1):
            y = BASE + 4 * step * rows
            share = bool(elements(BASE, b, t, 64, st) & elements(y, b, t, 64, st))
            assert share == (abs(rows) < n)
            assert conv(lib, p, BASE, y) == (INVALID if share else OK), (st, rows)
        for off in (n * step - 1, n * step + 1):
            y = BASE + 4 * off
            share = bool(elements(BASE, b, t, 64, st) & elements(y, b, t, 64, st))
            if share:
                assert conv(lib, p, BASE, y) == INVALID, (st, off)


def test_against_the_elements_they_share(lib):
    """Random tensors: what shares an element is refused, whatever its strides; with
    equal strides on both sides, column, token and sequence ranges pass."""
    g = np.random.default_rng(3)
    passed = 0
    for _ in range(4000):
        b, t, d = (int(v) for v in g.integers(1, 5, 3))
        st = []
        for _ in range(2):
            row = d + int(g.integers(0, 9))
            inner = row * int(g.integers(1, 3))
            outer = inner * int(g.integers(max(b, t), 12)) + int(g.integers(0, 2) * g.integers(0, 5))
            st.append((outer, inner) if g.random() < 0.6 else (inner, outer))
        if g.random() < 0.6:
            st[1] = st[0]
        p = gc.make_conv1d_problem(b, t, d, 2, 0, *st)
        y = BASE + 4 * int(g.integers(-80, 81))
        share = bool(elements(BASE, b, t, d, st[0]) & elements(y, b, t, d, st[1]))
        got = conv(lib, p, BASE, y)
        assert got in (OK, INVALID)
        if share:
            assert got == INVALID, (b, t, d, st, y - BASE)
        passed += got == OK
    assert passed > 500


def test_halves_of_a_long_buffer(lib):
    """Strides past 2^31."""
    st = (1 << 33, 4096)
    p = gc.make_conv1d_problem(3, 1 << 20, 4096, 4, 0, st, st)
    half = 4 * 4096 * (1 << 20)
    assert conv(lib, p, BASE, BASE + half) == OK
    assert conv(lib, p, BASE, BASE + half - 4) == INVALID and conv(lib, p, BASE, BASE + 4 * st[0]) == INVALID
