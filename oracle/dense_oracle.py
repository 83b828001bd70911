"""Float64 definitions of the dense products beside the routed experts: e4m3 codes with one scale per
block of 128 channels, and the gated feed-forward block with its backward pass."""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_values", "e4m3_round", "quant_fp8", "gemm_fp8", "act_and_slope", "gated_ff", "gated_ff_backward"]

E4M3_MAX = 448.0


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """Values of e4m3 codes (uint8): sign, four exponent bits with bias 7, three fraction bits; no infinities,
    all exponent and fraction bits set is NaN."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * np.exp2((e - 10).astype(np.float64)))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """uint8 codes of float64 values, |v| <= 448 after clamping, to nearest, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    table = e4m3_values(np.arange(127, dtype=np.uint8))          # 0 .. 448, ascending
    a = np.minimum(np.abs(v), E4M3_MAX)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(table[hi] == a, hi, code)
    code = np.where(np.isnan(v), 127, code)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quant_fp8(x: np.ndarray, block_rows: int = 1):
    """(codes uint8 [M][K], scales float32 [ceil(M / block_rows)][ceil(K / 128)]) of finite values."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    scales = np.zeros((-(-M // block_rows), -(-K // 128)), np.float32)
    codes = np.zeros((M, K), np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            s = np.float32(np.abs(x[at]).max() / E4M3_MAX)
            scales[i, j] = s
            quotient = (x[at] / float(s)).astype(np.float32) if s > 0 else np.zeros_like(x[at])
            codes[at] = e4m3_round(quotient)
    return codes, scales


def gemm_fp8(xq, xs, wq, ws, bias=None):
    """(y, S): the product and the sum of the magnitudes of its terms, float64 [M][N]."""
    K = xq.shape[1]
    x = e4m3_values(xq) * np.repeat(np.asarray(xs, np.float64), 128, axis=1)[:, :K]
    w = np.repeat(np.asarray(ws, np.float64), 128, axis=0)[:wq.shape[0]]
    w = e4m3_values(wq) * np.repeat(w, 128, axis=1)[:, :K]
    y, S = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, S = y + np.asarray(bias, np.float64), S + np.abs(np.asarray(bias, np.float64))
    return y, S


def act_and_slope(g: np.ndarray, act: str):
    g = np.asarray(g, np.float64)
    if act == "silu":
        p = 1.0 / (1.0 + np.exp(-g))
        return g * p, p + g * p * (1.0 - p)
    t = np.tanh(np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3))
    dt = (1.0 - t * t) * np.sqrt(2.0 / np.pi) * (1.0 + 3 * 0.044715 * g * g)
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * dt


def gated_ff(x, w, act: str):
    """(h [M][I], pre [M][2 I]) of x [M][H] and w [2 I][H]."""
    pre = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    I = pre.shape[1] // 2
    return act_and_slope(pre[:, :I], act)[0] * pre[:, I:], pre


def gated_ff_backward(dh, x, w, pre, act: str):
    """(dx [M][H], dw [2 I][H], dpre [M][2 I]) from the gradient of h."""
    dh, x, w, pre = (np.asarray(t, np.float64) for t in (dh, x, w, pre))
    I = dh.shape[1]
    a, s = act_and_slope(pre[:, :I], act)
    dpre = np.concatenate([dh * pre[:, I:] * s, dh * a], axis=1)
    return dpre @ w, dpre.T @ x, dpre
