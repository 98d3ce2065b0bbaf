"""Planner invariants of the sequence operators' other forms, on the CPU: the
host-only harness ``tests/harness/plan_seq_forms.cu`` built with nvcc.

* 8-bit product without TMA: tiles that cover the output, the teams' places, a shared
  tile's sums and the second ring within a block's shared memory and 1024-byte
  aligned, no more shared blocks than run at once;
* scan: the forward pass's second block for each slab where it pays, every ring of
  shared memory within a block's limit, as many blocks an SM as the launcher asks for."""
import json
import os
import shutil
import subprocess

import numpy as np
import pytest

from test_seq_plans import SMEM_BLOCK, matmul_problems

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SMEM_SM = 228 * 1024  # of an SM; 1 KB of a block's is the system's


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("forms") / "plan_seq_forms")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr", "-w",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "harness", "plan_seq_forms.cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [json.loads(x) for x in out.splitlines()]

    return run


@pytest.mark.parametrize("sms", [152, 148, 1])
def test_product_without_tma(plan, sms):
    g = np.random.default_rng(5)
    problems = [(max(1, M + int(g.integers(-7, 8))), max(1, N - int(g.integers(0, 7))), max(1, K - int(g.integers(1, 16))))
                for M, N, K in matmul_problems()] + [(1, 1, 1), (3, 5, 65536), (24, 40, 65531)]
    seen = set()
    for (M, N, K), p in zip(problems, plan([f"any {M} {N} {K} {sms}" for M, N, K in problems])):
        assert p["ok"], (M, N, K)
        assert p["BX"] % 16 == 0 and p["tiles_m"] * p["BX"] >= M > (p["tiles_m"] - 1) * p["BX"]
        assert p["tiles_n"] * 128 >= N > (p["tiles_n"] - 1) * 128 and p["tiles"] == p["tiles_m"] * p["tiles_n"]
        assert p["ksteps"] % 2 == 0 and p["ksteps"] * 64 >= K > (p["ksteps"] - 2) * 64
        assert p["ring"] >= p["places"] and p["ring"] % 1024 == 0 and p["wide"] == 4 * p["BX"] * 128
        assert 1024 + p["ring"] + p["wide"] + 1024 <= SMEM_BLOCK
        seen.add(p["split"])
        stages = p["ksteps"] // 2
        assert 1 <= p["split"] <= 8 and p["split"] * p["per"] >= stages > (p["split"] - 1) * p["per"]
        if p["split"] > 1:
            assert p["ring"] >= p["BX"] * 128 * 4 and p["tiles"] * p["split"] <= p["most"] <= sms
    assert seen == {1} if sms == 1 else len(seen) > 3


@pytest.mark.parametrize("sms", [152, 148, 1])
@pytest.mark.parametrize("bytes_", [2, 4])
def test_scan_forward_splits(plan, sms, bytes_):
    g = np.random.default_rng(6)
    problems = [(u, t) for u in (1, 75, 228, 229, 256, 266, 267, 304, 457) for t in (2, 64, 65, 512, 767, 768, 2048, 32768)]
    problems += [(int(2 ** g.uniform(0, 12)), int(2 ** g.uniform(1, 20))) for _ in range(300)]
    for (units, T), p in zip(problems, plan([f"scan {u} {t} {bytes_} {sms}" for u, t in problems])):
        ns = p["fwd"]
        assert 1 <= ns <= p["most"] <= 16 and (ns == 1 or (ns - 1) * 64 < T)
        if units * ns > 3 * sms:  # more blocks than places: one a slab, or the second of a slab
            assert ns == 1 or (ns == 2 and bytes_ == 2 and T >= 768 and 2 * units * 2 <= 7 * sms)
        if sms == 152 and T >= 768 and 229 <= units <= 266:
            assert ns == (2 if bytes_ == 2 else 1)
        if sms == 152 and 229 <= units and T < 768:
            assert ns == 1
        k = 0 if bytes_ == 2 else 1
        for ring, blocks in (("six", 2), ("eight", 1 if bytes_ == 2 else 2), ("forward", 3)):
            assert p[ring][k] <= SMEM_BLOCK and blocks * (p[ring][k] + 1024) <= SMEM_SM, ring
