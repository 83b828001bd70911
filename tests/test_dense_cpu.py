"""The e4m3 product and the gated feed-forward block without a GPU: the oracle against rationals and
differences, size queries, and the refusals that the library returns before any launch."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WS, ERR_DTYPE, ERR_OPTION = 0, -1, -2, -5, -7, -9, -10
P16, P8 = ctypes.c_void_p(16), ctypes.c_void_p(8)
BIG = 1 << 50


def _w(N=256, K=128, codes=16, scales=16):
    return cq._CWeightFp8(codes, scales, N, K)


def test_oracle_e4m3():
    every = np.arange(256, dtype=np.uint8)
    v = oracle.e4m3_values(every)
    t = torch.from_numpy(every.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    fine = ~np.isnan(v)
    assert (oracle.e4m3_round(v[fine]) == every[fine]).all()
    # halfway between neighbours: to the even code; off the half: to the nearer
    for c in range(126):
        lo, hi = v[c], v[c + 1]
        mid = (lo + hi) / 2
        assert oracle.e4m3_round(mid) == (c if c % 2 == 0 else c + 1)
        assert oracle.e4m3_round(np.nextafter(mid, 0)) == c and oracle.e4m3_round(np.nextafter(mid, 999)) == c + 1
        assert oracle.e4m3_round(-mid) == (c if c % 2 == 0 else c + 1) + 128
    assert oracle.e4m3_round(1e9) == 126 and oracle.e4m3_round(np.nan) & 127 == 127


@pytest.mark.parametrize("rows", [1, 128])
def test_oracle_quantiser(rows):
    rng = np.random.default_rng(rows)
    x = (rng.integers(-255, 256, (130, 144)) * 2.0 ** rng.integers(-9, 6, (130, 144))).astype(np.float32)
    x[:, :128][5 if rows == 1 else slice(0, 128)] = 0
    q, s = oracle.quant_fp8(x, rows)
    assert s.shape == (-(-130 // rows), 2)
    for i, j in ((0, 0), (5, 0), (5, 1), (129 // rows, 0), (129 // rows, 1)):
        if i >= s.shape[0]:
            continue
        part = x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
        amax = max(Fraction(float(abs(v))) for v in part.ravel())
        assert s[i, j] == np.float32(float(amax / 448))
        got = oracle.e4m3_values(q[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128])
        for a, b in zip(part.ravel()[:300], got.ravel()):
            if s[i, j] == 0:
                assert b == 0
                continue
            quotient = np.float32(float(a) / float(s[i, j]))
            table = oracle.e4m3_values(np.arange(127, dtype=np.uint8))
            assert abs(abs(b) - abs(quotient)) == np.abs(table - min(abs(quotient), np.float32(448))).min() or abs(quotient) > 448


def test_oracle_product_against_rationals():
    rng = np.random.default_rng(3)
    xq, wq = (rng.integers(0, 126, s).astype(np.uint8) | (rng.integers(0, 2, s) << 7).astype(np.uint8) for s in ((3, 144), (130, 144)))
    xs, ws = rng.normal(size=(3, 2)).astype(np.float32), rng.normal(size=(2, 2)).astype(np.float32)
    b = rng.normal(size=130).astype(np.float32)
    y, S = oracle.gemm_fp8(xq, xs, wq, ws, b)
    X, W = oracle.e4m3_values(xq), oracle.e4m3_values(wq)
    for m in range(3):
        for n in (0, 77, 128, 129):
            ref = Fraction(float(b[n]))
            for k in range(144):
                ref += Fraction(X[m, k]) * Fraction(W[n, k]) * Fraction(float(xs[m, k // 128])) * Fraction(float(ws[n // 128, k // 128]))
            assert abs(Fraction(y[m, n]) - ref) <= Fraction(S[m, n]) * 200 / 2 ** 53


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_gradients_against_differences(act):
    rng = np.random.default_rng(4)
    x, w, dh = rng.normal(size=(5, 16)), rng.normal(size=(24, 16)), rng.normal(size=(5, 12))
    dx, dw, _ = oracle.gated_ff_backward(dh, x, w, oracle.gated_ff(x, w, act)[1], act)
    loss = lambda a, b: float((oracle.gated_ff(a, b, act)[0] * dh).sum())
    e = 1e-5                                      # central differences: e^2 of the third derivative, 1e-16 / e of rounding
    for _ in range(20):
        vx, vw = rng.normal(size=x.shape), rng.normal(size=w.shape)
        d = (loss(x + e * vx, w + e * vw) - loss(x - e * vx, w - e * vw)) / (2 * e)
        ref = float((dx * vx).sum() + (dw * vw).sum())
        assert abs(d - ref) <= 1e-6 * (np.abs(dx * vx).sum() + np.abs(dw * vw).sum())


def test_quant_refusals():
    lib = cq.load_library()
    call = lambda x=P16, xd=1, M=4, K=128, rows=1, q=P16, s=P16: lib.cubic_quant_fp8(x, xd, M, K, rows, q, s, None)
    assert call(xd=0) == ERR_DTYPE and call(rows=0) == ERR_OPTION and call(rows=64) == ERR_OPTION
    for K in (0, -16, 8, 24, (1 << 20) + 16):
        assert call(K=K) == ERR_SHAPE
    assert call(M=-1) == ERR_SHAPE and call(M=1 << 24) == ERR_SHAPE and call(M=0, x=None, q=None, s=None) == OK
    assert call(x=None) == ERR_NULL and call(q=None) == ERR_NULL and call(s=None) == ERR_NULL
    assert call(x=P8) == ERR_ALIGN and call(q=P8) == ERR_ALIGN and call(s=P8) == ERR_ALIGN


def test_product_refusals():
    lib = cq.load_library()
    call = lambda w=_w(), M=4, xq=P16, xs=P16, b=None, y=P16, yd=0, ws=P16, n=BIG: lib.cubic_gemm_fp8(
        xq, xs, M, ctypes.byref(w), b, y, yd, ws, n, None)
    assert lib.cubic_gemm_fp8(P16, P16, 4, None, None, P16, 0, P16, BIG, None) == ERR_NULL
    for K in (0, -16, 8, 24, (1 << 20) + 16):
        assert call(_w(K=K)) == ERR_SHAPE
    assert call(_w(N=-1)) == ERR_SHAPE and call(M=-1) == ERR_SHAPE
    assert call(M=1 << 24) == ERR_SHAPE and call(_w(N=1 << 24)) == ERR_SHAPE
    assert call(yd=3) == ERR_DTYPE and call(yd=-1) == ERR_DTYPE
    assert call(M=0, xq=None) == OK and call(_w(N=0, codes=0)) == OK
    assert call(_w(codes=0)) == ERR_NULL and call(_w(scales=0)) == ERR_NULL
    assert call(xq=None) == ERR_NULL and call(xs=None) == ERR_NULL and call(y=None) == ERR_NULL
    assert call(_w(codes=8)) == ERR_ALIGN and call(_w(scales=8)) == ERR_ALIGN and call(ws=P8) == ERR_ALIGN
    assert call(b=P8) == ERR_ALIGN and call(xq=P8) == ERR_ALIGN and call(xs=P8) == ERR_ALIGN and call(y=P8) == ERR_ALIGN


def test_linear_refusals():
    lib = cq.load_library()
    call = lambda w=_w(), xd=1, M=8, x=P16, b=None, y=P16, ws=P16, n=BIG, yd=1: lib.cubic_linear_fp8(
        x, xd, M, ctypes.byref(w), b, y, yd, ws, n, None)
    assert call(xd=0) == ERR_DTYPE and call(yd=3) == ERR_DTYPE and call(_w(K=24)) == ERR_SHAPE
    assert call(x=None) == ERR_NULL and call(x=P8) == ERR_ALIGN and call(y=P8) == ERR_ALIGN and call(ws=P8) == ERR_ALIGN
    assert call(M=0, ws=None) == OK
    big = _w(N=4096, K=16384)
    need = lib.cubic_linear_fp8_workspace_bytes(200, 4096, 16384)
    assert need >= 200 * 16384 + 200 * 128 * 4
    assert call(big, M=200, ws=None) == ERR_WS and call(big, M=200, n=need - 1) == ERR_WS
    assert lib.cubic_linear_fp8_workspace_bytes(0, 5, 128) == 0 and lib.cubic_linear_fp8_workspace_bytes(5, 5, -1) == 0


def test_gated_refusals():
    lib = cq.load_library()
    call = lambda x=P16, w=P16, dt=1, M=4, H=64, I=64, act=0, h=P16, pre=None, ws=P16, n=BIG: lib.cubic_gated_ff(
        x, w, dt, M, H, I, act, h, pre, ws, n, None)
    for size in (0, -8, 4, 12, (1 << 20) + 8):
        assert call(H=size) == ERR_SHAPE and call(I=size) == ERR_SHAPE
    assert call(M=-1) == ERR_SHAPE and call(M=1 << 24) == ERR_SHAPE
    assert call(dt=0) == ERR_DTYPE and call(act=2) == ERR_OPTION and call(act=-1) == ERR_OPTION
    assert call(M=0, x=None, h=None) == OK
    assert call(x=None) == ERR_NULL and call(w=None) == ERR_NULL and call(h=None) == ERR_NULL
    for name in ("x", "w", "h", "pre", "ws"):
        assert call(**{name: P8}) == ERR_ALIGN
    need = lib.cubic_gated_ff_workspace_bytes(100, 4096, 64)
    if need:
        assert call(M=100, H=4096, ws=None) == ERR_WS and call(M=100, H=4096, n=need - 1) == ERR_WS


def test_backward_refusals():
    lib = cq.load_library()
    call = lambda dh=P16, x=P16, w=P16, pre=P16, dt=1, M=4, H=64, I=64, act=0, dx=P16, dw=P16, ws=P16, n=BIG: \
        lib.cubic_gated_ff_backward(dh, x, w, pre, dt, M, H, I, act, dx, dw, ws, n, None)
    assert call(H=12) == ERR_SHAPE and call(I=0) == ERR_SHAPE and call(dt=0) == ERR_DTYPE and call(act=9) == ERR_OPTION
    assert call(M=0, dw=None) == OK and call(dx=None, dw=None) == OK
    assert call(dh=None) == ERR_NULL and call(pre=None) == ERR_NULL and call(x=None) == ERR_NULL and call(w=None) == ERR_NULL
    for name in ("dh", "x", "w", "pre", "dx", "dw", "ws"):
        assert call(**{name: P8}) == ERR_ALIGN
    need = lib.cubic_gated_ff_backward_workspace_bytes(4, 64, 64)
    assert need >= 4 * 128 * 2
    assert call(ws=None) == ERR_WS and call(n=need - 1) == ERR_WS


def test_gated_fp8_refusals():
    lib = cq.load_library()
    call = lambda w=_w(), x=P16, xd=1, M=4, act=0, h=P16, hd=1, ws=P16, n=BIG: lib.cubic_gated_ff_fp8(
        x, xd, M, ctypes.byref(w), act, h, hd, ws, n, None)
    for N in (128, 255, 2 * 64, 384):
        assert call(_w(N=N)) == ERR_SHAPE
    assert call(_w(K=8)) == ERR_SHAPE and call(xd=0) == ERR_DTYPE and call(hd=0) == ERR_DTYPE and call(act=2) == ERR_OPTION
    assert call(M=0) == OK and call(_w(N=0)) == OK
    assert call(x=None) == ERR_NULL and call(h=None) == ERR_NULL and call(_w(codes=0)) == ERR_NULL
    assert call(x=P8) == ERR_ALIGN and call(h=P8) == ERR_ALIGN and call(ws=P8) == ERR_ALIGN and call(_w(scales=8)) == ERR_ALIGN
    need = lib.cubic_gated_ff_fp8_workspace_bytes(200, 16384, 2048)
    assert call(_w(4096, 16384), M=200, n=need - 1) == ERR_WS and call(_w(4096, 16384), M=200, ws=None) == ERR_WS


def test_binding_refusals():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((64, 64), dtype=torch.bfloat16)
    for call in (lambda: cq.cubic_gated_ff(x, w), lambda: cq.cubic_quant_fp8(x), lambda: cq.cubic_linear_fp8(x, None)):
        with pytest.raises(ValueError):               # host tensors
            call()
    with pytest.raises(TypeError):
        cq.cubic_quant_fp8(x.float())
    with pytest.raises(ValueError):
        cq._act("relu")
