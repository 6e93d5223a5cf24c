"""The training-step operators in a process that uses two devices: their
launchers against a stand-in for the CUDA runtime (tests/fake_runtime), since
kernels' attributes are per device and a handle per device shares the code. Runs
on the host; no GPU is touched."""
import os
import shutil
import subprocess

import pytest

from linear_cross_entropy_token_gb300 import build as flce_build

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_launchers_opt_in_on_every_device(tmp_path):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA toolkit headers")
    flce_build.build()
    exe = str(tmp_path / "two_devices")
    objects = [os.path.join(flce_build.BUILD, name + ".o") for name in ("flce_muon", "flce_muon_small", "flce_route")]
    cmd = ["g++", "-std=c++17", "-I", flce_build.CSRC, "-I", os.path.join(flce_build.ROOT, "include"),
           "-I", os.path.join(CUDA, "include"), os.path.join(HERE, "fake_runtime", "two_devices.cpp"), *objects, "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and " 0 refused" in r.stdout, r.stdout + r.stderr
