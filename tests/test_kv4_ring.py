"""Host-only check of the ring of bulk copies of the cache's attention (csrc/kv4_ring.cuh):
built from the same header with the host compiler and run on the CPU."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "exact_io_aware_26_gb300", "csrc")


def test_copies_under_way_are_known_when_a_wait_gives_up(tmp_path):
    exe = str(tmp_path / "ring_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-I", CSRC, os.path.join(HERE, "ring_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr + r.stdout
