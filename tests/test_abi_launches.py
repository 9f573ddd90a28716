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


def run(fake, *checks, lib=build.LIB, env=None):
    res = subprocess.run([sys.executable, os.path.join(HERE, "fake_hip_driver.py"), fake, lib,
                          *checks], capture_output=True, text=True, timeout=600, env=env)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "done" in res.stdout, out[-3000:]
    return out


@pytest.mark.parametrize("check", ["threads", "launches", "refusals"])
def test_few_token_entries(fake, check):
    """threads: a call's LDS limit holds between other threads' calls;
    launches: every size that is accepted launches within the limits;
    refusals: nothing is launched for what is refused."""
    run(fake, check)


def test_few_token_entries_under_host_asan(fake, tmp_path):
    """The same with the library's host code (argument checks, rules, launchers)
    under AddressSanitizer."""
    runtime = build.asan_runtime()
    if runtime is None:
        pytest.skip("clang's shared ASan runtime is not installed next to hipcc")
    lib = build.build_asan(tmp_path / "libmxfp4_asan.so")
    env = dict(os.environ, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0")
    out = run(fake, "threads", "launches", "refusals", lib=lib, env=env)
    assert "AddressSanitizer" not in out, out[-3000:]
    assert "asan_runtime_mapped 1" in out, out[-2000:]
