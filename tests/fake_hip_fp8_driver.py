"""Child-process driver of tests/test_abi_fp8.py (not a pytest module): the FP8
entry points over tests/c_abi/fake_hip.c, which launches nothing, at sizes over
the whole of what they accept. Stand-in pointers are never dereferenced.

Usage: python fake_hip_fp8_driver.py <fake_hip.so> <libmxfp4.so>
"""

import ctypes
import math
import random
import sys

P = 1 << 20
I64, VP, I32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
TOP = (1 << 31) - 256


def main():
    fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
    lib = ctypes.CDLL(sys.argv[2])
    lib.mxfp4_quantize_fp8.argtypes = [VP, I64, I64, I64, I64, I32, I32, VP, VP, VP]
    lib.mxfp4_quantize_fp8_2d.argtypes = [VP, I64, I64, I64, I64, I32, I32, VP, VP, VP, VP, VP]
    lib.mxfp4_gemm_fp8.argtypes = [VP, I32, VP, VP, VP, I32, I64, I64, I64, I64, I32, VP, VP]
    lib.mxfp4_gemm_fp8_swiglu_workspace.argtypes = [I64, I64, I64, ctypes.POINTER(I64)]
    lib.mxfp4_gemm_fp8_swiglu.argtypes = [VP, VP, VP, VP, I64, I64, I64, VP, VP, VP, VP, VP, VP]
    lib.mxfp4_swiglu_fp8_backward.argtypes = [VP, VP, I64, I64, I32, VP, VP, VP, VP, VP]
    assert lib.mxfp4_available() == 1
    count = ctypes.c_int.in_dll(fake, "fake_launches")
    count.value = 0
    rng = random.Random(3)

    def size(lo, hi, step=1):
        return step * round(math.exp(rng.uniform(math.log(lo / step), math.log(hi / step))))

    def launched(rc, what, n):
        assert rc == 0 and count.value == n, (what, rc, count.value)
        count.value = 0

    def shrunk(sizes, steps, fits):
        sizes = list(sizes)
        while not fits(*sizes):
            k = rng.randrange(len(sizes))
            sizes[k] = max(steps[k], sizes[k] // (2 * steps[k]) * steps[k])
        return sizes

    most = 1 << 40
    for _ in range(4000):
        M, K = shrunk((rng.choice([1, size(1, 64), size(1, TOP)]), size(16, 1 << 24, 16)), (1, 16),
                      lambda M, K: (M + 16) * K * 2 < most)
        rows, kind, scale = rng.choice([1, 128]), rng.randrange(2), rng.randrange(2)
        launched(lib.mxfp4_quantize_fp8(P, K, M, K, rows, kind, scale, P, P, None), (M, K), 1)
        M = min(M, 1 << 24)
        launched(lib.mxfp4_quantize_fp8_2d(P, K, M, K, rows, kind, scale, P, P, P, P, None),
                 (M, K), 1)
        M, N, K = shrunk((rng.choice([1, size(1, 1024), size(1, TOP)]), size(1, TOP),
                          size(16, 1 << 24, 16)), (1, 1, 16),
                         lambda M, N, K: M * K < most and N * K < most and M * N * 4 < most)
        rows = 128 if scale else rng.choice([1, 128])
        launched(lib.mxfp4_gemm_fp8(P, kind, P, P, P, scale, rows, M, N, K, rng.randrange(2), P,
                                    None), (M, N, K), 1)
        M, I, K = shrunk((rng.choice([1, size(1, 1024), size(1, TOP)]), size(128, 1 << 24, 128),
                          size(16, 1 << 24, 16)), (1, 128, 16),
                         lambda M, I, K: M * I * 4 < most and 2 * I * K < most and M * K < most)
        need = I64(-1)
        assert lib.mxfp4_gemm_fp8_swiglu_workspace(M, I, K, ctypes.byref(need)) == 0
        assert need.value in (0, 2 * M * I)
        launched(lib.mxfp4_gemm_fp8_swiglu(P, P, P, P, M, I, K, P, P, rng.choice([None, P]),
                                           rng.choice([None, P]), P if need.value else None, None),
                 (M, I, K), 2 if need.value else 1)
        M, I = shrunk((size(1, 1 << 24), I), (1, 128), lambda M, I: (M + 16) * I * 4 < most)
        launched(lib.mxfp4_swiglu_fp8_backward(P, P, M, I, kind, P, P, P, P, None), (M, I), 1)
    print("done", flush=True)


if __name__ == "__main__":
    main()
