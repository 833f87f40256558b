"""What the experts' entry points do on the host, seen without a GPU: tests/c_abi/experts_on_fake_device.c links them
against a stand-in for the CUDA runtime that reports any compute capability and counts launches."""
import os
import subprocess

import pytest
import torch

import combine_moe_route_02_gb300 as moe
import experts_ref as ref
from combine_moe_route_02_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, UNSUPPORTED = 0, 2
CALLS = {"moe_quantize_weight", "moe_expert_gemm", "moe_expert_wgrad", "moe_swiglu", "moe_swiglu_backward", "moe_layer",
         "moe_quantize_weight:widest"}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    _build.build()
    objects = [os.path.join(_build.BUILD, os.path.basename(s)[:-3] + ".o") for s in _build.sources()]
    if not all(os.path.exists(o) for o in objects):
        _build.build(force=True)
    out = tmp_path_factory.mktemp("fake_device")
    obj, exe = str(out / "fake.o"), str(out / "experts_on_fake_device")
    for cmd in (["gcc", "-std=c11", "-O1", "-Wall", "-Werror", "-fno-builtin", "-I", os.path.join(ROOT, "include"), "-c",
                 os.path.join(ROOT, "tests", "c_abi", "experts_on_fake_device.c"), "-o", obj],
                ["g++", "-o", exe, obj, *objects, "-ldl", "-lrt", "-lpthread"]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
    return exe


def run(program, *args):
    r = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
    out = {}
    for line in r.stdout.splitlines():
        name, status, launches, *grid = line.split()
        out[name] = (int(status), int(launches), tuple(map(int, grid)))
    return out


def test_one_launch_on_a_device_of_capability_10(program):
    got = run(program, 10)
    assert set(got) == CALLS and all(v[:2] == (OK, 1) for v in got.values()), got


@pytest.mark.parametrize("major", [8, 9, 12])
def test_other_devices_are_refused_before_a_launch(program, major):
    got = run(program, major)
    assert set(got) == CALLS and all(v[:2] == (UNSUPPORTED, 0) for v in got.values()), got


def test_the_widest_row_of_a_weight_has_a_grid(program):
    assert run(program, 10)["moe_quantize_weight:widest"] == (OK, 1, (2 ** 24, 1, 1))


@pytest.mark.gpu
def test_the_widest_row_of_a_weight():
    """2^31 - 8 columns, 4 GB: the first and the last block."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    moe.build()
    cols = 2 ** 31 - 8
    W = torch.zeros((1, cols), dtype=torch.bfloat16, device="cuda")
    ends = torch.arange(-60, 60, device="cuda").to(torch.bfloat16)      # the last block has 120 columns
    W[0, :120], W[0, -120:] = 2 * ends, ends
    q, s = moe.quantize_weight(W)
    assert s.shape == (1, 2 ** 24) and q.shape == (1, cols)
    for at, v in ((slice(0, 120), 2 * ends), (slice(cols - 120, cols), ends)):
        want_q, want_s = ref.encode_weight(v[None, None], "fp32")
        assert torch.equal(q[0, at], want_q[0, 0])
        assert s[0, 0 if at.start == 0 else -1] == want_s[0, 0, 0]
    assert not q[0, 128:cols - 120].any()
