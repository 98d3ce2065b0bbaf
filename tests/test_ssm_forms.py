"""Rules of the selective-block operators' kernels that a host can run: the harness f8_rules.cu, built with nvcc.  No
GPU needed."""
import json
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def harness(tmp_path_factory, name):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / name)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=compute_103a", "--expt-relaxed-constexpr", "-w",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(HERE, "harness", name + ".cu"), "-o", exe], check=True)

    def run(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [json.loads(x) for x in out.splitlines()]

    return run


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
