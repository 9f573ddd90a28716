"""What the library's host code asks of the HIP runtime, on a runtime that
launches nothing (tests/c_abi/fake_hip.c; CPU only)."""

import os
import subprocess
import sys

import pytest

from block_scaled_microscaling_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("fake") / "libfake_hip.so")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-fPIC", "-shared", "-isystem",
                    os.path.join(rocm, "include"), "-o", out,
                    os.path.join(HERE, "c_abi", "fake_hip.c")], check=True)
    return out


def run(fake, check):
    res = subprocess.run([sys.executable, os.path.join(HERE, "fake_hip_driver.py"), fake,
                          build.LIB, check], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "done" in res.stdout, (res.stdout + res.stderr)[-3000:]


def test_lds_limits_hold_between_threads(fake):
    run(fake, "threads")
