"""The limit on a kernel's dynamic shared memory only rises, on the CPU."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_smaller_size_cannot_take_a_larger_one_away(tmp_path):
    exe = str(tmp_path / "smem_attr")
    subprocess.run(["g++", "-std=c++17", "-pthread", os.path.join(HERE, "harness", "smem_attr.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True, timeout=60).stdout.split()
    assert out == ["200", "2", "0"], out
