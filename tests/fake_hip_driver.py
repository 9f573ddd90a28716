"""Child-process driver of tests/test_abi_launches.py (not a pytest module):
the library's few-token entry points over tests/c_abi/fake_hip.c, which
launches nothing. Stand-in pointers are never dereferenced.

Usage: python fake_hip_driver.py <fake_hip.so> <libmxfp4.so> <check>
"""

import ctypes
import sys

OK = 0
P = 1 << 20
I64, VP, I32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int


def load(fake_path, lib_path):
    fake = ctypes.CDLL(fake_path, mode=ctypes.RTLD_GLOBAL)
    lib = ctypes.CDLL(lib_path)
    lib.mxfp4_gemv.argtypes = [VP, I64, VP, VP, I64, I64, I64, I32, VP, VP]
    assert lib.mxfp4_available() == 1, "the fake device is not the one asked"
    return fake, lib


def gemv(lib, M, N, K, out=0):
    return lib.mxfp4_gemv(P, K, P, P, M, N, K, out, P, None)


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
    globals()[sys.argv[3]](*load(sys.argv[1], sys.argv[2]))
    print("done", flush=True)
