"""Forms of the selective-block operators that sizes are given to, and rules of their kernels that a host can run:
the harnesses plan_ssm.cu, plan_ssm_bwd.cu, f8_rules.cu and reads.cu, built with nvcc.  No GPU needed."""
import json
import os
import shutil
import subprocess

import numpy as np
import pytest

import f8_pairs as fp

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def harness(tmp_path_factory, name):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / name)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", "-Xcicc", "-O0", "--expt-relaxed-constexpr", "-w",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "harness", name + ".cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [json.loads(x) for x in out.splitlines()]

    return run


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return harness(tmp_path_factory, "plan_ssm")


@pytest.mark.parametrize("w_rows", [1, 128])
def test_sizes_of_pairs(plan, w_rows):
    sizes = [*fp.PAIRS, fp.EXACT, fp.STRIDED, *fp.CALLS]
    for size, p in zip(sizes, plan(["matmul %d %d %d %d %d" % (*q, w_rows, fp.SMS) for q in sizes])):
        assert p["ok"] and not p["swap"], size
    for size, p in zip(fp.OTHERS, plan(["matmul %d %d %d %d %d" % (*q, w_rows, fp.SMS) for q in fp.OTHERS])):
        assert p["ok"] and p["swap"], size


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return harness(tmp_path_factory, "f8_rules")


def test_a_ring_is_left_without_arrivals(rules):
    """At every barrier of a ring the phase of the last step that took its stage is waited for."""
    for stages in (2, 3, 4, 6, 12):
        for steps in range(0, 40):
            o, = rules([f"ring {steps} {stages} 0 0"])
            waited, st, phase = {}, o["stage"], o["phase"]
            for _ in range(o["from"], steps):
                waited[st] = phase
                st, phase = (0, phase ^ 1) if st + 1 == stages else (st + 1, phase)
            last = {step % stages: step // stages & 1 for step in range(steps)}
            assert waited == last, (stages, steps)


def test_rows_that_tma_may_store(rules):
    """Rows of y, their starts and their ends on 16 bytes: a store's last 16 bytes are written whole."""
    for es in (2, 4):
        for n in range(2096, 2113):
            for stride in (n, n + 1, 2112, 2120):
                for offset in (0, 8):
                    r, = rules([f"ymap {n} {stride} {es} {offset}"])
                    assert r["map"] == (n * es % 16 == 0 and stride * es % 16 == 0 and offset == 0), (es, n, stride, offset)


@pytest.fixture(scope="module")
def reads(tmp_path_factory):
    return harness(tmp_path_factory, "reads")


def words(first, have):
    """Halves that the aligned words around `have` 16-bit elements at `first` hold."""
    return (first // 2 * 2, (first + have + 1) // 2 * 2)


@pytest.mark.parametrize("B,T,D,gap", [(1, 1, 1, 0), (1, 5, 7, 0), (2, 17, 13, 0), (3, 33, 9, 2), (2, 16, 31, 5), (1, 40, 17, 1)])
def test_the_scan_reads_words_inside_its_tensors(reads, B, T, D, gap):
    """Chunks whose rows come by aligned words hold nothing outside the tensor, wherever it begins; the others come by
    elements."""
    pitch, cases = D + gap, []
    for b in range(B):
        cases += [(b, t) for t in range(0, T, 16)]
    ends = [r["ends"] for r in reads([f"chunk {b} {t} {B} {T} 0" for b, t in cases])]
    for off in (0, 1):
        start, stop = off, off + (B * T - 1) * pitch + D
        for (b, t), by_elements in zip(cases, ends):
            for at in range(t, min(t + 16, T)):
                for V in (2, 4, 8):
                    for e in range(0, D, V):
                        lo, hi = words(off + (b * T + at) * pitch + e, min(V, D - e))
                        assert by_elements or (lo >= start and hi <= stop), (off, b, at, V, e)
    assert not all(ends) or B * T <= 32


@pytest.mark.parametrize("rows,D,gap", [(1, 1, 0), (1, 40, 0), (2, 7, 0), (3, 41, 0), (4, 17, 3), (5, 8, 1)])
def test_the_norm_reads_words_inside_its_matrices(reads, rows, D, gap):
    V, pitch = 8, D + gap
    cases = [(r, e) for r in range(rows) for e in range(0, D, V)]
    ends = [r["ends"] for r in reads([f"vector {r} {e} {rows} {D} {V}" for r, e in cases])]
    for off in (0, 1):
        start, stop = off, off + (rows - 1) * pitch + D
        for (r, e), by_elements in zip(cases, ends):
            lo, hi = words(off + r * pitch + e, min(V, D - e))
            assert by_elements or (lo >= start and hi <= stop), (off, r, e)
    assert sum(ends) <= 2


def test_the_scans_backward_plans(tmp_path_factory):
    """Parts that cover the tokens at the saved states' distances, a workspace whose pieces follow one another, and
    grids within 31 bits wherever a problem is taken."""
    g = np.random.default_rng(3)
    small = [(1, 1, 1, 1, 1), (1, 32768, 2048, 16, 1), (8, 2048, 2048, 16, 1), (3, 1537, 700, 16, 2), (64, 1, 2048, 64, 8), (1, 1 << 33, 1, 1, 1)]
    small += [(int(2 ** g.uniform(0, 7)), int(2 ** g.uniform(0, 18)), int(2 ** g.uniform(0, 13)), int(g.integers(1, 65)), 1) for _ in range(300)]
    huge = [(1 << 31, 8, 64, 16, 1), (1, 1 << 36, 1, 1, 1), (1 << 20, 1 << 20, 1 << 10, 64, 1), (1 << 24, 1, 1 << 12, 64, 1 << 12)]
    plans = harness(tmp_path_factory, "plan_ssm_bwd")(["%d %d %d %d %d" % q for q in small + huge])
    assert not any(p["fits"] for p in plans[len(small):])
    for (B, T, D, N, G), p in zip(small, plans):
        assert p["fits"], (B, T, D, N, G)
        assert p["CC"] == 256 // p["lanes"] and p["lanes"] * 4 >= N
        assert p["tpg"] * p["CC"] >= D // G > (p["tpg"] - 1) * p["CC"]
        assert p["seg"] % (2 * p["chunk"]) == 0 and p["seg"] * p["S"] >= T > p["seg"] * (p["S"] - 1)
        assert p["cols"] == p["tpg"] * G * B * T * 8 * p["lanes"]
        assert p["ends"] == p["cols"] + B * p["S"] * D * (N + 2)
        assert p["sums"] == p["ends"] + (p["S"] - 1) * B * D * N and p["all"] == p["sums"] + (p["S"] - 1) * B * D
        assert B * p["tpg"] * G * p["S"] < 1 << 31 and p["sum_blocks"] < 1 << 31
