"""Host-side checks of the FP8 entry points of libmxfp4.so (no GPU work is
launched): exported symbols, refusals, the tensor layer's checks, and, over a
HIP runtime that launches nothing, the grids of all sizes that are accepted."""

import os
import re
import subprocess
import sys

import pytest
import torch

import block_scaled_microscaling_amd as mx
from block_scaled_microscaling_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(os.path.dirname(HERE), "include", "mxfp4_fp8.h")

OK, EINVAL, EUNSUPPORTED, EALIGN = 0, -1, -2, -4
P = 1 << 20             # stand-in pointer value: never dereferenced here
BIG = 1 << 62

QUANT = dict(x=P, ldx=256, M=4, K=256, rows=1, type=0, scale=0, codes=P, scales=P, stream=None)
QUANT2 = dict(x=P, ldx=256, M=4, K=256, rows=1, type=0, scale=0, codes=P, scales=P, codes_t=P,
              scales_t=P, stream=None)
GEMM = dict(a=P, type=0, sa=P, b=P, sb=P, scale=0, rows=128, M=4, N=33, K=256, out=0, C=P,
            stream=None)
SWIGLU = dict(a=P, sa=P, w=P, sw=P, M=4, I=256, K=64, codes=P, scales=P, act=None, gu=None, ws=P,
              stream=None)
BACK = dict(dact=P, gu=P, M=4, I=256, type=0, codes=P, scales=P, codes_t=P, scales_t=P,
            stream=None)
CALLS = {"quantize": (mx.mxfp4_quantize_fp8, QUANT), "quantize_2d": (mx.mxfp4_quantize_fp8_2d, QUANT2),
         "gemm": (mx.mxfp4_gemm_fp8, GEMM), "swiglu": (mx.mxfp4_gemm_fp8_swiglu, SWIGLU),
         "backward": (mx.mxfp4_swiglu_fp8_backward, BACK)}


def call(name, **kw):
    fn, args = CALLS[name]
    assert not set(kw) - set(args)
    return fn(*dict(args, **kw).values())


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp4_\w+)\s*\(", text)))
    assert names == ["mxfp4_gemm_fp8", "mxfp4_gemm_fp8_swiglu", "mxfp4_gemm_fp8_swiglu_workspace",
                     "mxfp4_quantize_fp8", "mxfp4_quantize_fp8_2d", "mxfp4_swiglu_fp8_backward"]
    for n in names:
        assert hasattr(mx.load_library(), n) and n in mx.__all__, n


SIZES = [dict(M=0), dict(M=-1), dict(M=1 << 31), dict(M=BIG)]
KS = [dict(K=0), dict(K=8), dict(K=-16), dict(K=24), dict(K=(1 << 24) + 16), dict(K=BIG)]
IS = [dict(I=0), dict(I=64), dict(I=-128), dict(I=192), dict(I=BIG), dict(I=(1 << 24) + 128)]


@pytest.mark.parametrize("name,bad", [
    (n, b) for n, bads in {
        "quantize": SIZES + KS + [dict(rows=0), dict(rows=2), dict(rows=64), dict(type=2),
                                  dict(type=-1), dict(scale=2), dict(ldx=255), dict(ldx=248),
                                  dict(ldx=260), dict(ldx=-256), dict(ldx=1 << 40),
                                  dict(M=(1 << 31) - 256, K=1 << 24, ldx=1 << 24)],
        "quantize_2d": SIZES + KS + [dict(rows=3), dict(type=5), dict(scale=-1), dict(ldx=248),
                                     dict(M=(1 << 24) + 1), dict(codes_t=None),
                                     dict(scales_t=None)],
        "gemm": SIZES + KS + [dict(N=0), dict(N=-1), dict(N=1 << 31), dict(type=2), dict(scale=2),
                              dict(rows=2), dict(rows=1, scale=1), dict(out=2), dict(out=-1),
                              dict(M=1 << 20, N=1 << 20), dict(M=1 << 17, K=1 << 23)],
        "swiglu": SIZES + KS + IS + [dict(ws=None), dict(M=1 << 20, I=1 << 18)],
        "backward": SIZES + IS + [dict(M=(1 << 24) + 1), dict(type=2), dict(M=1 << 24, I=1 << 15)],
    }.items() for b in bads])
def test_refuses(name, bad):
    if name.startswith("quantize") and "K" in bad and "ldx" not in bad:
        bad = dict(bad, ldx=1 << 24)
    assert call(name, **bad) == EINVAL


@pytest.mark.parametrize("name,arg", [
    (n, k) for n, (_, args) in CALLS.items() for k, v in args.items()
    if v == P and not (n == "swiglu" and k == "ws")])
def test_refuses_null(name, arg):
    assert call(name, **{arg: None}) == EINVAL


@pytest.mark.parametrize("name,bad", [
    ("quantize", dict(x=P + 8)), ("quantize", dict(codes=P + 8)),
    ("quantize", dict(scale=1, scales=P + 2)), ("quantize_2d", dict(codes_t=P + 4)),
    ("quantize_2d", dict(scale=1, scales_t=P + 1)), ("gemm", dict(a=P + 8)), ("gemm", dict(b=P + 1)),
    ("gemm", dict(C=P + 8)), ("gemm", dict(scale=1, sa=P + 2)), ("gemm", dict(scale=1, sb=P + 1)),
    ("swiglu", dict(a=P + 8)), ("swiglu", dict(w=P + 8)), ("swiglu", dict(codes=P + 4)),
    ("swiglu", dict(act=P + 2)), ("swiglu", dict(gu=P + 8)), ("swiglu", dict(ws=P + 4)),
    ("backward", dict(dact=P + 8)), ("backward", dict(gu=P + 2)), ("backward", dict(codes=P + 8)),
    ("backward", dict(codes_t=P + 8))])
def test_refuses_misaligned(name, bad):
    assert call(name, **bad) == EALIGN


@pytest.mark.parametrize("name,good", [
    ("quantize", dict(scales=P + 1)), ("quantize", dict(M=1, ldx=-3)),
    ("quantize_2d", dict(scales_t=P + 3)), ("gemm", dict(sa=P + 1, sb=P + 3)),
    ("gemm", dict(rows=1)), ("gemm", dict(scale=1)), ("swiglu", dict(act=P, gu=P, sw=P + 1)),
    ("backward", dict(scales=P + 1, scales_t=P + 1))])
def test_accepts_up_to_the_device(name, good):
    """Arguments that pass every check: refused for the missing device alone."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    assert call(name, **good) == EUNSUPPORTED


def test_workspace_sizes():
    assert mx.mxfp4_gemm_fp8_swiglu_workspace(4, 256, 64) == (OK, 2 * 4 * 256)
    assert mx.mxfp4_gemm_fp8_swiglu_workspace(16384, 14336, 4096) == (OK, 0)
    assert mx.mxfp4_gemm_fp8_swiglu_workspace(0, 256, 64)[0] == EINVAL
    assert mx.load_library().mxfp4_gemm_fp8_swiglu_workspace(4, 256, 64, None) == EINVAL


def test_tensor_layer_refuses_before_the_gpu():
    bf16 = torch.zeros((4, 256), dtype=torch.bfloat16)
    f8 = torch.zeros((4, 256), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        mx.quantize_fp8(bf16.float())
    with pytest.raises(ValueError, match="device tensor"):
        mx.quantize_fp8(bf16)
    with pytest.raises(ValueError, match="2-D"):
        mx.quantize_fp8_2d(bf16[0])
    with pytest.raises(TypeError, match="a must be torch.float8_e4m3fn or torch.float8_e5m2"):
        mx.gemm_fp8(bf16, s, f8, s)
    with pytest.raises(TypeError, match="a must be torch.float8_e4m3fn"):
        mx.gemm_fp8_swiglu(f8.view(torch.float8_e5m2), s, f8, s)
    with pytest.raises(ValueError, match="device tensor"):
        mx.gemm_fp8(f8, s, f8, s)
    with pytest.raises(TypeError, match="dact must be"):
        mx.swiglu_fp8_backward(f8, bf16)


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("fake") / "libfake_hip.so")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-fPIC", "-shared", "-isystem",
                    os.path.join(rocm, "include"), "-o", out,
                    os.path.join(HERE, "c_abi", "fake_hip.c")], check=True)
    return out


def test_every_accepted_size_launches_within_the_limits(fake):
    res = subprocess.run([sys.executable, os.path.join(HERE, "fake_hip_fp8_driver.py"), fake,
                          build.LIB], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0 and "done" in res.stdout, (res.stdout + res.stderr)[-3000:]
