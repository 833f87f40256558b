"""What the norms' and the joined products' entry points do on the host, seen without a GPU, as in test_experts_device.py:
tests/c_abi/norms_on_fake_device.c links them against a stand-in for the CUDA runtime."""
import os
import subprocess

import pytest

from combine_moe_route_02_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, UNSUPPORTED = 0, 2
LAUNCHES = {"moe_expert_swiglu": 1, "moe_expert_swiglu_backward": 1, "moe_rms_norm": 1, "moe_rms_norm:most": 1, "moe_rms_norm_backward": 2,
            "moe_rms_norm_backward:none": 1, "moe_grad_norm": 2, "moe_grad_norm:none": 1, "moe_clip_grad_norm": 2,
            "moe_clip_grad_norm:many": 4, "moe_grad_norm:empty": 2}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    _build.build()
    objects = [os.path.join(_build.BUILD, os.path.basename(s)[:-3] + ".o") for s in _build.sources()]
    if not all(os.path.exists(o) for o in objects):
        _build.build(force=True)
    out = tmp_path_factory.mktemp("fake_device")
    obj, exe = str(out / "fake.o"), str(out / "norms_on_fake_device")
    for cmd in (["gcc", "-std=c11", "-O1", "-Wall", "-Werror", "-Wno-unused-function", "-fno-builtin", "-I", os.path.join(ROOT, "include"), "-c",
                 os.path.join(ROOT, "tests", "c_abi", "norms_on_fake_device.c"), "-o", obj],
                ["g++", "-o", exe, obj, *objects, "-ldl", "-lrt", "-lpthread"]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
    return exe


def run(program, major):
    r = subprocess.run([program, str(major)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
    out = {}
    for line in r.stdout.splitlines():
        name, status, launches, *grid = line.split()
        out[name] = (int(status), int(launches), tuple(map(int, grid)))
    return out


def test_launches_on_a_device_of_capability_10(program):
    got = run(program, 10)
    assert {k: v[1] for k, v in got.items()} == LAUNCHES and all(v[0] == OK for v in got.values()), got
    assert got["moe_rms_norm:most"][2] == (2 ** 31 - 1, 1, 1)


@pytest.mark.parametrize("major", [8, 9, 12])
def test_other_devices_are_refused_before_a_launch(program, major):
    got = run(program, major)
    assert set(got) == set(LAUNCHES) and all(v[:2] == (UNSUPPORTED, 0) for v in got.values()), got
