"""The int8 product without a GPU: the oracle against integers, size queries, and the refusals that
the library returns before any launch."""
import ctypes
from fractions import Fraction

import numpy as np

import dequant_gemm_amd as cq
import oracle

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_DTYPE = 0, -1, -2, -5, -7, -9
P16, P8 = ctypes.c_void_p(16), ctypes.c_void_p(8)


def _w(N=32, K=64, codes=16, scales=16):
    return cq._CWeightI8(codes, scales, N, K)


def test_oracle_against_rationals():
    rng = np.random.default_rng(1)
    xq = rng.integers(-128, 128, (3, 24)).astype(np.int8)
    wq = rng.integers(-128, 128, (5, 24)).astype(np.int8)
    sx, sw, b = (rng.normal(size=n).astype(np.float32) for n in (3, 5, 5))
    y = oracle.gemm_w8a8(xq, sx, wq, sw, b)
    for m in range(3):
        for n in range(5):
            I = sum(int(a) * int(c) for a, c in zip(xq[m], wq[n]))
            ref = Fraction(I) * Fraction(float(sx[m])) * Fraction(float(sw[n])) + Fraction(float(b[n]))
            assert abs(Fraction(float(y[m, n])) - ref) <= abs(ref) * Fraction(1, 2 ** 50) + Fraction(1, 2 ** 60)


def test_oracle_quantiser():
    """The rule by rationals: one rounding for the scale, one for each quotient, ties to even."""
    rn32 = lambda v: np.float32(float(v))                    # exact products of two fp32 numbers fit a double
    inv = np.float32(1.0 / 127.0)
    assert inv == np.float32(float(Fraction(1, 127)))
    rng = np.random.default_rng(2)
    x = (rng.integers(-255, 256, (20, 24)) * 2.0 ** rng.integers(-6, 6, (20, 1))).astype(np.float32)
    x[3] = 0
    q, s = oracle.quant_w8a8(x)
    for m in range(20):
        amax = max(Fraction(float(abs(v))) for v in x[m])
        assert s[m] == rn32(amax * Fraction(float(inv)))
        for k in range(24):
            if s[m] == 0:
                assert q[m, k] == 0
                continue
            quot = np.float32(float(x[m, k]) / float(s[m]))  # 53 bits hold enough of the quotient to round once more
            assert q[m, k] == max(-127, min(127, round(Fraction(float(quot)))))


def test_refusals():
    lib = cq.load_library()
    call = lambda w=_w(), M=4, xq=P16, xs=P16, b=None, y=P16, yd=0: lib.cubic_gemm_w8a8(
        xq, xs, M, ctypes.byref(w), b, y, yd, None)
    assert lib.cubic_gemm_w8a8(P16, P16, 4, None, None, P16, 0, None) == ERR_NULL
    for K in (0, -8, 12, 131072):
        assert call(_w(K=K)) == ERR_SHAPE
    assert call(_w(N=-1)) == ERR_SHAPE and call(M=-1) == ERR_SHAPE and call(M=1 << 31) == ERR_SHAPE
    assert call(M=1 << 24) == ERR_SHAPE and call(_w(N=1 << 24)) == ERR_SHAPE
    assert call(yd=2) == ERR_DTYPE
    assert call(M=0) == OK and call(_w(N=0, codes=0)) == OK             # no-ops
    assert call(_w(codes=0)) == ERR_NULL and call(xq=None) == ERR_NULL and call(xs=None) == ERR_NULL
    assert call(y=None) == ERR_NULL
    assert call(_w(codes=8)) == ERR_ALIGN and call(_w(scales=8)) == ERR_ALIGN
    assert call(b=P8) == ERR_ALIGN and call(xq=P8) == ERR_ALIGN and call(y=P8) == ERR_ALIGN


def test_linear_refusals_and_workspace():
    lib = cq.load_library()
    need = lib.cubic_linear_w8a8_workspace_bytes
    assert need(4, 8192) == 0 and need(0, 64) == 0 and need(4, 0) == 0
    assert need(5, 72) == 512 + 256 and need(1, 8200) == 8448 + 256
    call = lambda w=_w(), xd=1, M=8, x=P16, ws=P16, n=1 << 20, yd=1: lib.cubic_linear_w8a8(
        x, xd, M, ctypes.byref(w), None, P16, yd, ws, n, None)
    assert call(xd=0) == ERR_DTYPE and call(yd=2) == ERR_DTYPE
    assert call(_w(K=60)) == ERR_SHAPE
    assert call(x=None) == ERR_NULL and call(x=P8) == ERR_ALIGN
    assert call(ws=None) == ERR_WS and call(n=700) == ERR_WS and call(ws=P8) == ERR_ALIGN
    assert call(M=0, ws=None) == OK
