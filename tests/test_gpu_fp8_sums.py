"""Sums of the e4m3 products, where a sum in fewer bits than fp32's shows: blocks whose largest products cancel
each other, and blocks with terms of 2^-18 beside one of 2^5.

All terms are whole multiples of one power of two and no partial sum reaches 2^24 of them, whatever the order, so fp32
sums are exact and so are the sums over blocks under scales that are powers of two: results are the exact value rounded
once, bit for bit. The gated form: gate and up exact, the activation within 2^-18 |g|, half a step of the type."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
OUTS = [torch.bfloat16, torch.float16, torch.float32]


def _codes(values):
    """e4m3 codes of values that are codes' values."""
    return torch.from_numpy(oracle.e4m3_round(values)).to(DEV).view(torch.float8_e4m3fn)


def _operands(kind, M, N, K, seed):
    """(x values [M][K], w values [N][K], xs, ws) of code values and scales that are powers of two."""
    rng = np.random.default_rng(seed)
    kb = -(-K // 128)
    x, w = np.empty((M, K)), np.empty((N, K))
    for b in range(kb):
        k0, n = b * 128, min(128, K - b * 128)
        if kind == "cancel":
            # up to eight products of 448 * 448 and as many of -448 * 448 (200704, 1.6 million at most in a
            # partial sum), the others at most 8 * 8: sums below 2^24
            at = rng.permutation(n)
            pairs = 1 + int(rng.integers(0, min(8, n // 4)))
            x[:, k0:k0 + n] = rng.integers(1, 9, (M, n))
            w[:, k0:k0 + n] = rng.integers(-8, 9, (N, n))
            x[:, k0 + at[:2 * pairs]] = 448.0
            w[:, k0 + at[:pairs]], w[:, k0 + at[pairs:2 * pairs]] = 448.0, -448.0
        else:
            # terms of 1 to 9 times 2^-18 and one of 32: below 2^24 times 2^-18
            x[:, k0:k0 + n] = rng.integers(1, 4, (M, n)) * 2.0 ** -9
            w[:, k0:k0 + n] = rng.integers(1, 4, (N, n)) * 2.0 ** -9
            at = int(rng.integers(0, n))
            x[:, k0 + at], w[:, k0 + at] = 8.0, 4.0
    # "cancel": a block's sum is at most 128 * 64, with its scales' product (2^-4 to 1) 2^17 of the smallest unit: the sum
    # over 17 blocks stays below 2^24 units. "small": scales of one
    lo = (-2, 1) if kind == "cancel" else (0, 1)
    xs = np.exp2(rng.integers(*lo, (M, kb))).astype(np.float32)
    ws = np.exp2(rng.integers(*lo, (-(-N // 128), kb))).astype(np.float32)
    return x, w, xs, ws


def _scaled(v, scales, rows):
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, axis=0)[:v.shape[0]], 128, axis=1)
    return v * s[:, :v.shape[1]]


def _bits(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


# few rows (whole, quantised in chunks, beside one), then tiles of every shape and slices of the contraction
SIZES = [(1, 300, 528), (3, 6200, 272), (5, 129, 2064), (16, 1003, 1936), (24, 4500, 400), (32, 260, 144), (33, 2050, 400), (40, 6200, 528), (64, 300, 2048),
         (65, 64, 2064), (100, 1003, 1040), (130, 520, 144), (300, 6000, 208), (515, 2050, 528), (700, 384, 2064), (1030, 2050, 144), (2051, 4113, 272), (4101, 4113, 144)]


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("kind", ["cancel", "small"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_is_exact(M, N, K, kind, out):
    if kind == "small" and K > 256:
        K = 256 if K % 128 == 0 else 144
    say(f"gemm_fp8 exact sums M={M} N={N} K={K} {kind} {out}")
    x, w, xs, ws = _operands(kind, M, N, K, M + N)
    if kind == "small" and K > 128:                   # the second block has a scale of zero
        ws[:, 1] = 0.0
    ref = torch.from_numpy(_scaled(x, xs, 1) @ _scaled(w, ws, 128).T)
    want = ref.float()
    assert torch.equal(want.double(), ref)            # representable: what follows rounds once
    want = want.to(out)
    scales = [torch.from_numpy(s).to(DEV) for s in (xs, ws)]
    weight = cq.Fp8Weight(_codes(w), scales[1])
    y = cq.cubic_gemm_fp8(_codes(x), scales[0], weight, out_dtype=out).cpu()
    assert torch.equal(_bits(y), _bits(want)), (y != want).double().mean()
    if kind == "cancel":                              # every block holds 448: the quantiser gives these codes
        rows = torch.from_numpy(_scaled(x, xs, 1)).to(torch.bfloat16).to(DEV)
        y = cq.cubic_linear_fp8(rows, weight, out_dtype=out).cpu()
        assert torch.equal(_bits(y), _bits(want)), (y != want).double().mean()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(1, 528, 256), (4, 272, 2304), (9, 2064, 128), (17, 400, 2304), (33, 528, 384), (64, 1040, 128), (65, 2064, 128), (130, 272, 512),
                                   (515, 528, 1024), (1030, 144, 1024), (2051, 272, 2048), (4101, 144, 2048)])
def test_gated_block_is_exact(M, H, I, out, act):
    say(f"gated_ff_fp8 exact sums M={M} H={H} I={I} {act} {out}")
    x, w, xs, ws = _operands("cancel", M, 2 * I, H, M + I)
    xs, ws = xs * np.float32(2.0 ** -6), ws * np.float32(2.0 ** -6)      # gates of a few units
    rows = torch.from_numpy(_scaled(x, xs, 1)).to(torch.bfloat16).to(DEV)
    weight = cq.Fp8Weight(_codes(w), torch.from_numpy(ws).to(DEV))
    h = cq.cubic_gated_ff_fp8(rows, weight, act=act, out_dtype=out).double().cpu().numpy()
    ref, pre = oracle.gated_ff(_scaled(x, xs, 1), _scaled(w, ws, 128), act)
    tol = 2.0 ** -18 * np.abs(pre[:, :I] * pre[:, I:])
    tol = tol * (1 + HALF[out]) + HALF[out] * np.abs(ref) + 2.0 ** -25
    assert (np.abs(h - ref) <= tol).all(), (np.abs(h - ref) / tol).max()
