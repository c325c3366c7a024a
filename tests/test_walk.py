"""How a product's workgroups find their tiles, replayed on the host (`host_walk.cpp`)
with the index arithmetic that the kernels use: no tile outside what launch and
workspace are sized for, whatever the offsets hold."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "two_sided_gptq_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


def test_every_tile_lies_in_the_workspace(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is missing")
    drv = tmp_path / "walk"
    subprocess.run([HIPCC, "--cuda-host-only", "-x", "hip", "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "host_walk.cpp"),
                    "-o", str(drv)], check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(drv)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "walk checks passed" in r.stdout, r.stderr
