"""GPU parity of the dense products at sizes where each tile shape is the quickest, whole and cut into slices,
against the oracle, within the tolerances of the operators' own tests; and the e4m3 linear call with few rows,
which it quantises in one way or another."""
import pytest
import torch

import dequant_gemm_amd as cq
from tests import test_gpu_fp8 as fp8
from tests import test_gpu_gated_ff as ff
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
ACT = {torch.bfloat16: "silu", torch.float16: "gelu_tanh"}


# the largest tile of the forward product first, its sliced ones last
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(2051, 1032, 2056), (2051, 72, 2056), (4101, 72, 2056), (1300, 1032, 1032), (700, 4104, 264), (300, 1544, 520)])
def test_forward_tiles(M, H, I, dtype):
    say(f"gated_ff tiles M={M} H={H} I={I} {dtype}")
    x, w, _ = ff._data(M + H, M, H, I, dtype)
    h, guard = ff._guarded((M, I), dtype)
    pre, guard_p = ff._guarded((M, 2 * I), torch.float32)
    cq.cubic_gated_ff(x, w, act=ACT[dtype], out=h, pre=pre)
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_p).all())
    ff._check_h(h, pre, x, w, ACT[dtype], dtype)


# both gradients in one launch where that is quickest (256 x 256 down to 64 x 64), then each in its own
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(2500, 8200, 1544), (2051, 4104, 1032), (515, 4104, 520), (3000, 136, 136), (2051, 136, 136), (300, 136, 136), (4101, 72, 2056),
                                   (2051, 4104, 136), (2051, 2056, 136), (3000, 1032, 136), (515, 1032, 2056), (1030, 136, 2056),
                                   (300, 2056, 2056), (300, 1032, 2056), (1300, 1032, 1032), (3000, 1032, 264), (5000, 40, 4104)])
def test_backward_tiles(M, H, I, dtype):
    say(f"gated_ff_backward tiles M={M} H={H} I={I} {dtype}")
    x, w, dh = ff._data(M + I, M, H, I, dtype)
    pre = torch.randn((M, 2 * I), generator=torch.Generator(device=DEV).manual_seed(I), device=DEV)
    dx, guard = ff._guarded((M, H), dtype)
    dw, guard_w = ff._guarded((2 * I, H), dtype)
    cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], dx=dx, dw=dw)
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_w).all())
    ff._check_grads(dx, dw, dh, x, w, pre, ACT[dtype], dtype)
    one, _ = cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], need_dw=False)
    _, two = cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], need_dx=False)
    ff._check_grads(one, two, dh, x, w, pre, ACT[dtype], dtype)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(2051, 4113, 1168), (4101, 4113, 656), (2051, 4113, 144), (3000, 3001, 144), (4101, 4113, 144), (2051, 2050, 144), (1030, 2050, 144), (515, 2050, 528),
                                   (130, 520, 144), (130, 1003, 2064)])
def test_fp8_tiles(M, N, K, out):
    say(f"gemm_fp8 tiles M={M} N={N} K={K} {out}")
    xq, xs, w, b = fp8._data(M + N, M, N, K, bias=bool(N & 1))
    y, guard = fp8._guarded((M, N), out)
    cq.cubic_gemm_fp8(xq, xs, w, bias=b, out=y, out_dtype=out)
    assert bool(torch.isnan(guard).all())
    fp8._check(y, xq, xs, w, b, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(2051, 1168, 2048), (2051, 144, 2048), (4101, 144, 2048), (2051, 144, 1024), (1030, 144, 1024), (515, 528, 1024)])
def test_fp8_block_tiles(M, H, I, out):
    ff.test_fp8_block(M, H, I, ACT[out], out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(2, 64, 40960), (5, 40, 16400), (6, 129, 8208), (8, 7000, 4112), (16, 1003, 2048), (16, 6144, 2560), (17, 300, 5776),
                                   (31, 2050, 1040), (33, 1003, 1936), (48, 4096, 2048), (64, 2050, 1536), (64, 37, 16)])
def test_linear_of_few_rows_is_quantiser_and_product(M, N, K, dtype):
    """Bit for bit, with blocks of zeros, of the type's smallest values and of non-finite ones."""
    say(f"linear_fp8 few rows M={M} N={N} K={K} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = fp8._acts(g, M, K, dtype)
    x[0, :min(K, 256)] = 0
    x[0, 0] = -0.0
    x[1, :min(K, 128)] = -2.0 ** -133 if dtype == torch.bfloat16 else -2.0 ** -24
    if M > 4:
        x[3], x[4, 7], x[2, K - 1] = 0, float("nan"), -float("inf")
    _, _, w, b = fp8._data(N, 8, N, K, bias=True)
    xq, xs = cq.cubic_quant_fp8(x)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        want = cq.cubic_gemm_fp8(xq, xs, w, bias=b, out_dtype=out)
        y, guard = fp8._guarded((M, N), out)
        assert cq.cubic_linear_fp8_workspace_bytes(M, N, K) >= cq.cubic_gemm_fp8_workspace_bytes(M, N, K)
        cq.cubic_linear_fp8(x, w, bias=b, out=y, out_dtype=out)
        assert bool(torch.isnan(guard).all())
        bits = torch.int32 if out == torch.float32 else torch.int16
        assert torch.equal(torch.isnan(y), torch.isnan(want)) and bool(torch.isfinite(y[:2]).all())
        assert torch.equal(torch.where(torch.isnan(y), 0, y).view(bits), torch.where(torch.isnan(want), 0, want).view(bits))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(5, 528, 384), (8, 4112, 2176), (16, 1040, 1152), (17, 528, 256), (31, 1040, 1024), (37, 528, 1024), (64, 1040, 128)])
def test_fp8_block_of_few_rows(M, H, I, out):
    ff.test_fp8_block(M, H, I, ACT[out], out)
