"""Child-process driver of tests/test_abi_launches.py (not a pytest module):
the library's few-token entry points over tests/c_abi/fake_hip.c, which
launches nothing. Stand-in pointers are never dereferenced.

Usage: python fake_hip_driver.py <fake_hip.so> <libmxfp4.so> <check>...
"""

import ctypes
import math
import random
import sys

OK, EINVAL, EALIGN = 0, -1, -4
P = 1 << 20
I64, VP, I32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int


def load(fake_path, lib_path):
    fake = ctypes.CDLL(fake_path, mode=ctypes.RTLD_GLOBAL)
    lib = ctypes.CDLL(lib_path)
    size = ctypes.POINTER(I64)
    lib.mxfp4_gemv.argtypes = [VP, I64, VP, VP, I64, I64, I64, I32, VP, VP]
    lib.mxfp4_moe_route_workspace.argtypes = [I64, I64, I64, size]
    lib.mxfp4_moe_route.argtypes = [VP, I64, VP, I64, I64, I64, I64, I32, VP, VP, VP, VP]
    lib.mxfp4_moe_workspace.argtypes = [I64, I64, I64, I64, size]
    lib.mxfp4_moe.argtypes = [VP, I64, VP, VP, VP, VP, VP, VP, I64, I64, I64, I64, I64, I32, VP,
                              VP, VP]
    assert lib.mxfp4_available() == 1, "the fake device is not the one asked"
    return fake, lib


def gemv(lib, M, N, K, out=0):
    return lib.mxfp4_gemv(P, K, P, P, M, N, K, out, P, None)


def route(lib, T, H, E, k, renorm=1, ws=P):
    return lib.mxfp4_moe_route(P, H, P, T, H, E, k, renorm, P, P, ws, None)


def moe(lib, T, H, I, E, k, out=0, ws=P):
    return lib.mxfp4_moe(P, H, P, P, P, P, P, P, T, H, I, E, k, out, P, ws, None)


def workspace(fn, *sizes):
    n = I64(-1)
    return fn(*sizes, ctypes.byref(n)), n.value


def launches(fake, lib):
    """Sizes over the whole of what the entries accept: every call launches
    within the limits of a grid, a workgroup and its LDS."""
    rng = random.Random(1)
    count = ctypes.c_int.in_dll(fake, "fake_launches")

    def size(lo, hi, step=1):
        return step * round(math.exp(rng.uniform(math.log(lo / step), math.log(hi / step))))

    def launched(rc, what, least, most):
        assert rc == OK and least <= count.value <= most, (what, rc, count.value)
        count.value = 0

    count.value = 0
    for _ in range(4000):
        M = rng.choice([1, size(1, 64), size(1, 65535 * 16)])
        N, K = size(1, (1 << 31) - 1), size(32, 1 << 24, 32)
        while N * K // 2 >= 1 << 40 or M * K * 2 >= 1 << 40 or M * N * 4 >= 1 << 40:
            N, K = max(1, N // 2), max(32, K // 64 * 32)
        launched(gemv(lib, M, N, K, rng.randrange(2)), ("gemv", M, N, K), 1, 1)
        E = size(1, 1024)
        T, H, k = size(1, 65535), size(8, 1 << 24, 8), rng.randint(1, min(E, 32))
        while T * H * 2 >= 1 << 40:
            H = max(8, H // 16 * 8)
        rc, need = workspace(lib.mxfp4_moe_route_workspace, T, H, E)
        assert rc == OK and need >= 0
        launched(route(lib, T, H, E, k, ws=P if need else None), ("route", T, H, E, k),
                 2 if need else 1, 2 if need else 1)
        k = rng.randint(1, 32)
        T, H, I = size(1, 1024 // k), size(32, 1 << 20, 32), size(32, 1 << 20, 32)
        E = size(1, 1024)
        while E * H * I >= 1 << 40:
            H = max(32, H // 64 * 32)
        rc, need = workspace(lib.mxfp4_moe_workspace, T, H, I, k)
        assert rc == OK and need >= 4 * T * k * I
        launched(moe(lib, T, H, I, E, k, rng.randrange(2)), ("moe", T, H, I, E, k), 2, 3)


def refusals(fake, lib):
    """Nothing is launched for an argument that is refused."""
    count = ctypes.c_int.in_dll(fake, "fake_launches")
    count.value = 0
    big = 1 << 62
    assert lib.mxfp4_gemv(None, 64, P, P, 2, 2, 64, 0, P, None) == EINVAL
    assert lib.mxfp4_gemv(P + 8, 64, P, P, 2, 2, 64, 0, P, None) == EALIGN
    assert lib.mxfp4_gemv(P, 60, P, P, 2, 2, 64, 0, P, None) == EINVAL
    for M, N, K in [(0, 2, 64), (2, 0, 64), (2, 2, 48), (big, 2, 64), (2, big, 64), (2, 2, big)]:
        assert gemv(lib, M, N, K) == EINVAL
    assert gemv(lib, 2, 2, 64, out=2) == EINVAL
    for T, H, E, k in [(0, 64, 8, 2), (2, 60, 8, 2), (2, 64, 0, 1), (2, 64, 8, 9), (2, 64, 64, 33),
                       (big, 64, 8, 2), (2, big, 8, 2), (2, 64, big, 2), (2, 64, 8, big)]:
        assert route(lib, T, H, E, k) == EINVAL
    assert route(lib, 300, 64, 8, 2, ws=None) == EINVAL
    assert route(lib, 2, 64, 8, 2, renorm=2) == EINVAL
    for T, H, I, E, k in [(0, 64, 64, 8, 2), (2, 48, 64, 8, 2), (2, 64, 48, 8, 2), (2, 64, 64, 0, 2),
                          (2, 64, 64, 8, 33), (1025, 64, 64, 8, 1), (big, 64, 64, 8, 2),
                          (2, big, 64, 8, 2), (2, 64, big, 8, 2), (2, 64, 64, big, 2),
                          (2, 64, 64, 8, big), (1 << 32, 64, 64, 8, 1 << 32)]:
        assert moe(lib, T, H, I, E, k) == EINVAL
    assert moe(lib, 2, 64, 64, 8, 2, ws=None) == EINVAL
    assert moe(lib, 2, 64, 64, 8, 2, ws=P + 8) == EALIGN
    assert lib.mxfp4_moe_workspace(2, 64, 64, 2, None) == EINVAL
    assert lib.mxfp4_moe_route_workspace(2, 64, 8, None) == EINVAL
    assert count.value == 0


def threads(fake, lib):
    """A kernel's LDS limit is the process's: a call of a short K (whose waves,
    and LDS, are few) from another thread must not lower it between another
    call's set and launch."""
    M, N = 16, 6200
    for out in (0, 1):
        assert gemv(lib, M, N, 8192, out) == OK
        most = ctypes.c_size_t.in_dll(fake, "fake_most_lds").value
        assert most > 65536, most               # the kernel that needs the limit raised
        inner = []
        between = ctypes.CFUNCTYPE(None)(lambda: inner.append(gemv(lib, M, N, 256, out)))
        hook = ctypes.c_void_p.in_dll(fake, "fake_between")
        hook.value = ctypes.cast(between, ctypes.c_void_p).value
        rc = gemv(lib, M, N, 8192, out)
        hook.value = None
        assert rc == OK and inner in ([], [OK]), (rc, inner)
        assert gemv(lib, M, N, 8192, out) == OK


if __name__ == "__main__":
    both = load(sys.argv[1], sys.argv[2])
    for check in sys.argv[3:]:
        globals()[check](*both)
    with open("/proc/self/maps") as f:
        print("done, asan_runtime_mapped", int("libclang_rt.asan" in f.read()), flush=True)
