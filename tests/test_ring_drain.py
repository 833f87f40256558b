"""The copies that the norm's gradient has under way when one of its waits ran out: tests/c_abi/ring_drain.cc stops its ring
at every point and checks the waits that csrc/bulk_ring.cuh has it make before it leaves."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_drain")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "combine_moe_route_02_gb300", "csrc"),
           os.path.join(ROOT, "tests", "c_abi", "ring_drain.cc"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def test_every_copy_has_landed_wherever_the_ring_stops(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "6776 cases, 0 wrong\n", r.stdout


def test_the_model_sees_waits_that_go_by_the_loop_instead(program):
    r = subprocess.run([program, "by_count"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 1 and "wrong" in r.stdout
