"""Host-side checks of the few-token entry points of libmxfp4.so (no GPU work
is launched): exported symbols, refusals and the tensor layer's checks."""

import os
import re

import pytest
import torch

import block_scaled_microscaling_amd as mx

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "mxfp4_fewtoken.h")

OK, EINVAL, EUNSUPPORTED, EALIGN = 0, -1, -2, -4
P = 1 << 20             # stand-in pointer value: never dereferenced here

GEMV = dict(x=P, ldx=256, codes=P, scales=P, M=4, N=33, K=256, dtype=mx.OUT_BF16, y=P, stream=None)
ROUTE = dict(x=P, ldx=64, router=P, T=4, H=64, E=8, k=2, renorm=1, ids=P, weights=P, ws=P,
             stream=None)
MOE = dict(x=P, ldx=64, ids=P, weights=P, w13=P, w13_s=P, w2=P, w2_s=P, T=4, H=64, I=96, E=8, k=2,
           dtype=mx.OUT_FP32, y=P, ws=P, stream=None)


def gemv(**kw):
    return mx.mxfp4_gemv(*dict(GEMV, **kw).values())


def route(**kw):
    return mx.mxfp4_moe_route(*dict(ROUTE, **kw).values())


def moe(**kw):
    return mx.mxfp4_moe(*dict(MOE, **kw).values())


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mxfp4_\w+)\s*\(", text)))
    assert names == ["mxfp4_gemv", "mxfp4_moe", "mxfp4_moe_route", "mxfp4_moe_route_workspace",
                     "mxfp4_moe_workspace"]
    for n in names:
        assert hasattr(mx.load_library(), n) and n in mx.__all__, n


@pytest.mark.parametrize("bad", [
    dict(M=0), dict(M=-1), dict(M=65535 * 16 + 1), dict(N=0), dict(N=-5), dict(N=1 << 31),
    dict(K=0), dict(K=16), dict(K=48), dict(K=-32), dict(K=(1 << 24) + 32), dict(dtype=2),
    dict(dtype=-1), dict(ldx=255), dict(ldx=248), dict(ldx=260), dict(ldx=0), dict(ldx=-256),
    dict(ldx=1 << 40), dict(N=(1 << 31) - 1, K=1 << 24, ldx=1 << 24),
    dict(M=1 << 19, N=(1 << 31) - 1, dtype=mx.OUT_FP32),
    dict(x=None), dict(codes=None), dict(scales=None), dict(y=None)])
def test_gemv_refuses(bad):
    assert gemv(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(x=P + 8), dict(codes=P + 8), dict(y=P + 2)])
def test_gemv_refuses_misaligned(bad):
    assert gemv(**bad) == EALIGN


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=65536), dict(H=0), dict(H=60), dict(H=(1 << 24) + 8), dict(E=0),
    dict(E=1025), dict(k=0), dict(k=9), dict(k=-1), dict(E=64, k=33), dict(renorm=2),
    dict(renorm=-1), dict(ldx=56), dict(ldx=68), dict(ldx=0),
    dict(x=None), dict(router=None), dict(ids=None), dict(weights=None),
    dict(ws=None, H=4096, ldx=4096, E=128)])
def test_route_refuses(bad):
    assert route(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(x=P + 8), dict(router=P + 4), dict(ids=P + 2),
                                 dict(weights=P + 1), dict(ws=P + 8)])
def test_route_refuses_misaligned(bad):
    assert route(**bad) == EALIGN


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=513), dict(T=1 << 40), dict(T=33, k=32), dict(k=0), dict(k=33, T=1),
    dict(H=0), dict(H=48), dict(H=(1 << 20) + 32), dict(I=0), dict(I=80), dict(I=(1 << 20) + 32),
    dict(E=0), dict(E=1025), dict(E=1024, H=1 << 20, I=1 << 20, ldx=1 << 20), dict(dtype=3),
    dict(ldx=56), dict(ldx=68), dict(x=None), dict(ids=None), dict(weights=None), dict(w13=None),
    dict(w13_s=None), dict(w2=None), dict(w2_s=None), dict(y=None), dict(ws=None)])
def test_moe_refuses(bad):
    assert moe(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(x=P + 8), dict(ids=P + 2), dict(weights=P + 2),
                                 dict(w13=P + 8), dict(w2=P + 4), dict(y=P + 1), dict(ws=P + 8)])
def test_moe_refuses_misaligned(bad):
    assert moe(**bad) == EALIGN


def test_one_row_needs_no_row_stride():
    want = EUNSUPPORTED
    if mx.mxfp4_available():
        pytest.skip("a gfx950 device is present; stand-in pointers must not reach it")
    assert gemv(M=1, ldx=0) == route(T=1, ldx=0) == moe(T=1, ldx=0) == want
    assert gemv() == route() == moe() == want
    # Scales are byte-addressed.
    assert gemv(scales=P + 1) == moe(w13_s=P + 3, w2_s=P + 1) == want


def test_workspace_sizes():
    # A size that one launch handles needs none, and then takes NULL.
    assert mx.mxfp4_moe_route_workspace(4, 64, 8) == (OK, 0)
    if not mx.mxfp4_available():
        assert route(ws=None) == EUNSUPPORTED
    rc, n = mx.mxfp4_moe_route_workspace(64, 4096, 128)
    assert rc == OK and n >= 64 * 128 * 8
    rc, n = mx.mxfp4_moe_workspace(32, 2048, 768, 8)
    assert rc == OK and n >= 32 * 8 * 768 * 4
    for args in [(0, 64, 8), (65536, 64, 8), (4, 64, 0), (4, 64, 1025), (4, 0, 8), (4, 60, 8),
                 (4, (1 << 24) + 8, 8)]:
        assert mx.mxfp4_moe_route_workspace(*args)[0] == EINVAL
    for args in [(0, 64, 32, 1), (4, 64, 33, 1), (4, 64, 0, 1), (4, 64, 32, 0), (4, 64, 32, 33),
                 (1025, 64, 32, 1), (4, 48, 32, 1), (4, 0, 32, 1), (4, (1 << 20) + 32, 32, 1)]:
        assert mx.mxfp4_moe_workspace(*args)[0] == EINVAL


def test_tensor_layer_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    c = torch.zeros((8, 32), dtype=torch.uint8)
    s = torch.zeros((8, 2), dtype=torch.uint8)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for fn, rest in [(mx.gemv, (c, s)), (mx.moe_route, (x, 2)),
                     (mx.moe, (ids, ids.float(), c[None], s[None], c[None], s[None]))]:
        with pytest.raises(ValueError):
            fn(x, *rest)                        # not on a device
        with pytest.raises(ValueError):
            fn(x[0], *rest)                     # not 2-D
        with pytest.raises(TypeError):
            fn(x.float(), *rest)
        with pytest.raises(TypeError):
            fn([1.0], *rest)
