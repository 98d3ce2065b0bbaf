"""Planner invariants of the sequence operators, on the CPU: the host-only harness
``tests/harness/plan_seq.cu`` built with nvcc.

* 8-bit product: tiles that cover the output, shared memory within the block's
  limit, TMA boxes within 256 rows, stage bases 1024-byte aligned, a ring in which
  a stage always belongs to the same teams, accumulators and the teams' operand
  stages apart in tensor memory;
* scan: no more blocks in a cluster than the map buffers hold, none without
  tokens, shared memory within the limit."""
import json
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SMEM_BLOCK = 232448


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / "plan_seq")
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr", "-w",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "harness", "plan_seq.cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [json.loads(x) for x in out.splitlines()]

    return run


def matmul_problems():
    g = np.random.default_rng(1)
    fixed = [(9, 1, 16), (8192, 8192, 2048), (197, 5000, 2048), (1 << 20, 64, 64), (16, 1 << 21, 64), (100, 100, 65536)]
    rand = [(int(2 ** g.uniform(3.2, 14)), int(2 ** g.uniform(0, 14)), 16 * int(2 ** g.uniform(0, 9))) for _ in range(300)]
    return fixed + rand


@pytest.mark.parametrize("sms", [152, 148, 1])
def test_matmul_plans(plan, sms):
    problems = matmul_problems()
    for (M, N, K), p in zip(problems, plan([f"matmul {M} {N} {K} {sms}" for M, N, K in problems])):
        assert p["ok"], (M, N, K)
        assert p["BX"] % 16 == 0 and 16 <= p["BX"] <= p["max_bx"] <= 256
        assert p["tiles_m"] * p["BX"] >= M > (p["tiles_m"] - 1) * p["BX"]
        assert p["tiles_n"] * 128 >= N > (p["tiles_n"] - 1) * 128 and p["tiles"] == p["tiles_m"] * p["tiles_n"]
        assert p["ksteps"] % 2 == 0 and p["ksteps"] * 64 >= K > (p["ksteps"] - 2) * 64
        assert p["raw_bytes"] == (128 + p["BX"]) * 128 and p["wide_bytes"] == p["BX"] * 128
        assert p["raw_bytes"] % 1024 == 0 and p["wide_bytes"] % 1024 == 0
        assert p["teams"] % 2 == 0 and p["raw_stages"] >= 2 and p["raw_stages"] % (p["teams"] // 2) == 0
        assert 1024 + p["raw_stages"] * p["raw_bytes"] + p["teams"] * p["wide_bytes"] + 1024 <= SMEM_BLOCK
        assert p["threads"] <= 1024
        assert p["max_bx"] + p["BX"] <= p["wide_col"] and p["wide_col"] + 32 * p["teams"] <= 512


def test_matmul_refuses_unaligned_rows(plan):
    assert not plan(["matmul 100 100 40 152"])[0]["ok"]


@pytest.mark.parametrize("sms", [152, 148, 1])
def test_scan_splits(plan, sms):
    g = np.random.default_rng(2)
    problems = [(32, 32768, 64), (1, 2, 64), (66, 1537, 64), (256, 2048, 64)]
    problems += [(int(2 ** g.uniform(0, 12)), int(2 ** g.uniform(1, 20)), int(g.choice([32, 64, 128]))) for _ in range(300)]
    for (units, T, tokens), p in zip(problems, plan([f"scan {u} {t} {k} {sms}" for u, t, k in problems])):
        for ns in (p["fwd"], p["bwd"]):
            assert 1 <= ns <= p["most"] <= 16
            assert ns == 1 or (ns - 1) * tokens < T
        assert p["fwd"] >= p["bwd"]
        assert max(p["smem"]) <= SMEM_BLOCK


def ring(steps, stages, teams, warps, seed):
    """The barriers of the product's rings under a random interleaving: a copied
    stage is two steps, step s is team s % teams', waits look at one parity bit.
    Raises where an agent works on a stage that is not its step's."""
    import random

    class Bar:
        def __init__(self, n):
            self.n, self.left, self.phase = n, n, 0

        def arrive(self):
            self.left -= 1
            if self.left == 0:
                self.left, self.phase = self.n, self.phase + 1

        def ready(self, parity):
            return self.phase & 1 != parity

    r = random.Random(seed)
    raw_full, raw_empty = [Bar(1) for _ in range(stages)], [Bar(2 * warps) for _ in range(stages)]
    wide_full, wide_empty = [Bar(warps) for _ in range(teams)], [Bar(1) for _ in range(teams)]
    raw, wide, done, flying, issued = [None] * stages, [None] * teams, [], [], []

    def producer():
        for q in range(steps // 2):
            while q >= stages and not raw_empty[q % stages].ready((q // stages - 1) & 1):
                yield
            flying.append(q)
            yield

    def copies():
        while True:
            if flying and r.random() < 0.3:
                q = flying.pop(r.randrange(len(flying)))
                raw[q % stages] = q
                raw_full[q % stages].arrive()
            yield

    def team(t):
        at, raw_parity, wide_parity = t // 2, 0, 1
        for s in range(t, steps, teams):
            while not raw_full[at].ready(raw_parity):
                yield
            while s >= teams and not wide_empty[t].ready(wide_parity):
                yield
            assert raw[at] == s // 2
            yield
            assert raw[at] == s // 2
            wide[t] = s
            raw_empty[at].arrive()
            wide_full[t].arrive()
            wide_parity ^= 1
            at += teams // 2
            if at >= stages:
                at, raw_parity = at - stages, raw_parity ^ 1
            yield

    def issuer():
        for s in range(steps):
            while not wide_full[s % teams].ready((s // teams) & 1):
                yield
            assert wide[s % teams] == s
            issued.append(s)
            yield

    def tensor_cores():
        while True:
            if issued and r.random() < 0.4:
                s = issued.pop(0)
                assert wide[s % teams] == s
                done.append(s)
                wide_empty[s % teams].arrive()
            yield

    agents = [producer(), copies(), issuer(), tensor_cores()] + [team(t) for t in range(teams) for _ in range(warps)]
    for _ in range(400000):
        k = r.randrange(len(agents))
        try:
            next(agents[k])
        except StopIteration:
            agents.pop(k)
        if len(done) == steps:
            return done
    raise AssertionError("stuck")


@pytest.mark.parametrize("stages", [2, 4, 6, 12])
def test_ring_protocol(stages):
    for seed in range(20):
        assert ring(32, stages, 4, 3, seed) == list(range(32))


def test_ring_protocol_needs_a_multiple_of_the_pairs():
    """With three copied stages a team skips phases and takes an old one for its
    own: what the planner's rounding prevents."""
    with pytest.raises(AssertionError):
        for seed in range(50):
            ring(32, 3, 4, 3, seed)


@pytest.mark.parametrize("sms", [152, 148, 1])
def test_shared_tiles(plan, sms):
    """Blocks that share a tile: each has a part of K, all run at once, and a
    block's sums fit where its copied stages were."""
    problems = matmul_problems() + [(16, 2048, 2048), (64, 1024, 4096), (128, 2048, 2048), (16, 128, 65536), (9, 1, 16)]
    seen = set()
    for (M, N, K), p in zip(problems, plan([f"share {M} {N} {K} {sms}" for M, N, K in problems])):
        seen.add(p["split"])
        assert 1 <= p["split"] <= p["most"] <= 8
        stages = p["ksteps"] // 2
        assert p["split"] * p["per"] >= stages > (p["split"] - 1) * p["per"]
        if p["split"] > 1:
            assert p["tiles"] * p["split"] <= p["room"] <= sms and p["BX"] * 128 * 4 <= p["ring"]
    assert seen == {1} if sms == 1 else len(seen) > 3
