"""Where the e4m3 linear call quantises its rows inside the product: the same result as the two calls by
themselves, on both sides of every border of that choice, and the gated form over the same rows."""
import pytest
import torch

import dequant_gemm_amd as cq
from tests import test_gpu_fp8 as fp8
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
# (rows, weight rows, channels, quantised inside): rows staged whole, rows in chunks, too many rows, values or weight rows
CASES = [(4, 300, 4112, True), (4, 5000, 32768, True), (4, 300, 32784, False), (5, 300, 4112, True), (8, 4096, 4096, True), (8, 1003, 1936, True), (8, 4096, 4112, False),
         (5, 4352, 528, False), (9, 300, 528, False), (16, 1003, 1936, False), (37, 1003, 1936, False), (5, 300, 16, True),
         (1, 8192, 528, True), (1, 8193, 528, False), (4, 8448, 272, False), (16, 9000, 144, False)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,inside", CASES)
def test_linear_on_both_sides(M, N, K, inside, dtype):
    say(f"linear_fp8 M={M} N={N} K={K} inside={inside} {dtype}")
    assert (cq.cubic_linear_fp8_workspace_bytes(M, N, K) == 0) == inside
    x = fp8._acts(torch.Generator(device=DEV).manual_seed(M + K), M, K, dtype)
    _, _, w, b = fp8._data(N, 1, N, K, bias=True)
    for out in (torch.float32, torch.bfloat16):
        y, guard = fp8._guarded((M, N), out)
        cq.cubic_linear_fp8(x, w, bias=b, out=y, out_dtype=out)
        assert bool(torch.isnan(guard).all())
        assert torch.equal(y, cq.cubic_gemm_fp8(*cq.cubic_quant_fp8(x), w, bias=b, out_dtype=out))
    if N % 256 == 0:
        h = cq.cubic_gated_ff_fp8(x, w, out_dtype=torch.float16)
        spread = lambda t, rows: t.repeat_interleave(rows, 0).repeat_interleave(128, 1)  # noqa: E731
        q, s = cq.cubic_quant_fp8(x)
        xd, wd = q.double() * spread(s, 1)[:, :K], w.codes.double() * spread(w.scales, 128)[:N, :K]
        pre, e = xd @ wd.t(), (K + 4 * s.shape[1]) * 2.0 ** -24 * (xd.abs() @ wd.abs().t())
        g, u, eg, eu = pre[:, :N // 2], pre[:, N // 2:], e[:, :N // 2], e[:, N // 2:]
        ref = g * torch.sigmoid(g) * u
        # fp32 sums, carried through |act'| <= 1.13; the activation within 2^-18 |g|; half a step
        tol = 1.13 * eg * (u.abs() + eu) + g.abs() * eu + 2.0 ** -18 * (g * u).abs()
        tol = tol * (1 + 2.0 ** -11) + 2.0 ** -11 * ref.abs() + 2.0 ** -25
        assert bool(((h.double() - ref).abs() <= tol).all())
