"""Workspaces of the e4m3 calls: nothing is asked for that no kernel reads, and where the size query gives 0 a call
without a workspace succeeds."""
import ctypes

import pytest
import torch

import dequant_gemm_amd as cq

DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
# rows that the streaming kernel takes, whatever the result's type: up to 16 beside up to 8192 weight rows, to 32 beside up to
# 4096, to 64 beside those and up to 4096 channels
FEW = [(1, 6144, 7168), (16, 8192, 7168), (17, 1003, 1936), (32, 4096, 7168), (33, 1003, 1936), (37, 1003, 1936), (64, 4096, 4096)]
align = lambda n: -(-n // 256) * 256  # noqa: E731


@pytest.mark.parametrize("M,N,K", FEW)
def test_few_rows_ask_for_no_slices(M, N, K):
    assert cq.cubic_gemm_fp8_workspace_bytes(M, N, K) == 0
    staged = align(M * K) + align(M * -(-K // 128) * 4)
    assert cq.cubic_linear_fp8_workspace_bytes(M, N, K) in (0, staged)
    if N % 256 == 0:
        assert cq.cubic_gated_ff_fp8_workspace_bytes(M, K, N // 2) == cq.cubic_linear_fp8_workspace_bytes(M, N, K)


def test_gated_form_of_few_rows():
    assert cq.cubic_gated_ff_fp8_workspace_bytes(32, 7168, 2048) == align(32 * 7168) + align(32 * 56 * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", FEW + [(1, 300, 528), (4, 512, 1040), (8, 512, 1040), (16, 256, 528), (40, 512, 272)])
def test_calls_without_a_workspace(M, N, K, out):
    print(f"[gpu-case] fp8 without a workspace M={M} N={N} K={K} {out}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    xq, xs = cq.cubic_quant_fp8(x)
    w = cq.Fp8Weight(*cq.cubic_quant_fp8(torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16), block_rows=128))
    lib, st = cq.load_library(), torch.cuda.current_stream().cuda_stream
    cw = cq._CWeightFp8(w.codes.data_ptr(), w.scales.data_ptr(), N, K)
    ref = cq.cubic_gemm_fp8(xq, xs, w, out_dtype=out)
    y = torch.empty_like(ref)
    assert lib.cubic_gemm_fp8(xq.data_ptr(), xs.data_ptr(), M, ctypes.byref(cw), None, y.data_ptr(), DT[out], None, 0, st) == 0
    assert torch.equal(y, ref)
    if cq.cubic_linear_fp8_workspace_bytes(M, N, K) == 0:
        y.zero_()
        assert lib.cubic_linear_fp8(x.data_ptr(), 1, M, ctypes.byref(cw), None, y.data_ptr(), DT[out], None, 0, st) == 0
        assert torch.equal(y, ref)
    if N % 256 == 0 and out != torch.float32 and cq.cubic_gated_ff_fp8_workspace_bytes(M, K, N // 2) == 0:
        h = torch.empty((M, N // 2), dtype=out, device="cuda")
        assert lib.cubic_gated_ff_fp8(x.data_ptr(), 1, M, ctypes.byref(cw), 0, h.data_ptr(), DT[out], None, 0, st) == 0
        assert torch.equal(h, cq.cubic_gated_ff_fp8(x, w, out_dtype=out))
