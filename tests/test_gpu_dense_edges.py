"""Edges of the dense products: offsets beyond 4 GiB, the longest rows, slices of the contraction with odd widths,
activations quantised inside and outside the product, non-finite codes in fp32 results, a workspace that graphs share
in turn, inputs that are one tensor. Tolerances as in the two operators' own tests."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say
from tests.test_gpu_fp8 import _acts, _check, _data, _guarded, _np
from tests.test_gpu_gated_ff import F, _check_grads, _check_h
from tests.test_gpu_gated_ff import _data as _ff_data

pytestmark = pytest.mark.gpu
NAN = float("nan")
bits = lambda t: t.view({2: torch.int16, 4: torch.int32}[t.element_size()])  # noqa: E731


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 20, 33, 64, 100])
def test_linear_is_quantiser_and_product_bit_for_bit(M, out):
    say(f"linear_fp8 = quant + gemm M={M} {out}")
    g = torch.Generator(device=DEV).manual_seed(M)
    for N, K in ((260, 144), (1003, 1936), (5000, 4112), (40, 32768)):
        x = _acts(g, M, K, torch.float16)
        _, _, w, b = _data(M, 1, N, K, bias=True)
        y = cq.cubic_linear_fp8(x, w, bias=b, out_dtype=out)
        z = cq.cubic_gemm_fp8(*cq.cubic_quant_fp8(x), w, bias=b, out_dtype=out)
        assert torch.equal(bits(y), bits(z)), (N, K)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(70, 333, 8192), (100, 1003, 4096), (130, 130, 16384), (17, 4500, 1040), (40, 5000, 528), (64, 17, 8208)])
def test_slices_and_odd_widths(M, N, K, out):
    say(f"fp8 slices M={M} N={N} K={K} {out}")
    xq, xs, w, b = _data(M + N, M, N, K, bias=True)
    y, guard = _guarded((M, N), out)
    need = cq.cubic_gemm_fp8_workspace_bytes(M, N, K)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    cq.cubic_gemm_fp8(xq, xs, w, bias=b, out=y, out_dtype=out, workspace=ws[:max(need, 1)])
    assert bool(torch.isnan(guard).all()) and bool((ws[need:] == 0xFF).all())
    _check(y, xq, xs, w, b, out)


@pytest.mark.parametrize("M", [1, 20, 90, 300])
def test_nan_codes_in_fp32_results(M):
    say(f"fp8 NaN codes fp32 M={M}")
    xq, xs, w, _ = _data(M, M, 270, 528)
    clean = cq.cubic_gemm_fp8(xq, xs, w)
    codes, rows = w.codes.clone(), xq.clone()
    codes.view(torch.uint8)[200, 17] = 0xFF
    rows.view(torch.uint8)[M // 2, 300] = 0x7F
    got = cq.cubic_gemm_fp8(rows, xs, cq.Fp8Weight(codes, w.scales))
    bad = torch.zeros((M, 270), dtype=torch.bool, device=DEV)
    bad[:, 200], bad[M // 2] = True, True
    assert torch.equal(torch.isnan(got), bad)
    assert torch.equal(bits(got)[~bad], bits(clean)[~bad])


@pytest.mark.parametrize("M", [2, 70])
def test_longest_rows(M):
    K = 1 << 20
    say(f"K = 2^20, M={M}")
    xq, xs, w, _ = _data(M, M, 24, K)
    _check(cq.cubic_gemm_fp8(xq, xs, w), xq, xs, w, None, torch.float32)
    _check(cq.cubic_gemm_fp8(xq, xs, w, out_dtype=torch.bfloat16), xq, xs, w, None, torch.bfloat16)
    x, w16, dh = _ff_data(M, M, K, 8, torch.bfloat16)
    h, pre = cq.cubic_gated_ff(x, w16, save_pre=True)
    _check_h(h, pre, x, w16, "silu", torch.bfloat16)
    dx, dw = cq.cubic_gated_ff_backward(dh, x, w16, pre)
    _check_grads(dx, dw, dh, x, w16, pre, "silu", torch.bfloat16)


@pytest.mark.parametrize("M,H,I", [(70, 8192, 136), (130, 4096, 520), (100, 16384, 72), (66, 136, 8200), (9000, 8, 8), (8, 8, 9000)])
def test_gated_slices_and_long_sides(M, H, I):
    say(f"gated slices M={M} H={H} I={I}")
    x, w, dh = _ff_data(M + I, M, H, I, torch.float16)
    sizes = cq.cubic_gated_ff_workspace_bytes(M, H, I), cq.cubic_gated_ff_backward_workspace_bytes(M, H, I)
    ws = [torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes]
    h, pre = cq.cubic_gated_ff(x, w, act="gelu_tanh", save_pre=True, workspace=ws[0][:max(sizes[0], 1)])
    _check_h(h, pre, x, w, "gelu_tanh", torch.float16)
    dx, dw = cq.cubic_gated_ff_backward(dh, x, w, pre, act="gelu_tanh", workspace=ws[1][:sizes[1]])
    _check_grads(dx, dw, dh, x, w, pre, "gelu_tanh", torch.float16)
    assert all(bool((t[n:] == 0xFF).all()) for t, n in zip(ws, sizes))


def test_fp8_beyond_4_gib():
    """Codes of 4.6 GB, as activations and as the weight: rows at both ends are right, all others zero."""
    say("fp8 codes beyond 4 GiB")
    R, K = 70000, 65536
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = [0, 1, 33000, 65535, 65537, R - 2, R - 1]
    big = torch.zeros((R, K), dtype=torch.uint8, device=DEV)
    few, fs = cq.cubic_quant_fp8(_acts(g, len(rows), K))
    big[rows] = few.view(torch.uint8)
    codes = big.view(torch.float8_e4m3fn)
    scales = torch.ones((R, K // 128), device=DEV)
    scales[rows] = fs
    xq, xs, w, _ = _data(3, 70, 40, K)
    y = cq.cubic_gemm_fp8(codes, scales, w)
    _check(y[rows], few, fs, w, None, torch.float32)
    assert sorted(torch.nonzero(y.any(dim=1)).flatten().tolist()) == rows
    blocks = torch.full((-(-R // 128), K // 128), 0.5, device=DEV)
    for M in (2, 70):
        y = cq.cubic_gemm_fp8(xq[:M], xs[:M].contiguous(), cq.Fp8Weight(codes, blocks))
        part = cq.Fp8Weight(few, torch.full((1, K // 128), 0.5, device=DEV))
        _check(y[:, rows], xq[:M], xs[:M], part, None, torch.float32)
        assert sorted(torch.nonzero(y.any(dim=0)).flatten().tolist()) == rows


def test_gated_beyond_4_gib():
    """Activations and their gradient of 4.4 GB, rows apart from the chosen ones zero."""
    say("gated block beyond 4 GiB")
    M, H, I = 270336, 8192, 16
    x, w, dh = _ff_data(2, 6, H, I, torch.bfloat16)
    rows = [0, 131072, 262143, 262144, M - 2, M - 1]
    bx = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    bd = torch.zeros((M, I), dtype=torch.bfloat16, device=DEV)
    bx[rows], bd[rows] = x, dh
    h, pre = cq.cubic_gated_ff(bx, w, save_pre=True)
    _check_h(h[rows], pre[rows], x, w, "silu", torch.bfloat16)
    assert not bool(h[2:131072].any())
    dx, dw = cq.cubic_gated_ff_backward(bd, bx, w, pre)
    ref_x, ref_w, _ = oracle.gated_ff_backward(F(dh), F(x), F(w), F(pre[rows]), "silu")
    _check_grads(dx[rows], None, dh, x, w, pre[rows], "silu", torch.bfloat16)
    _check_grads(None, dw, dh, x, w, pre[rows], "silu", torch.bfloat16)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert not bool(dx[keep].any())


def test_graphs_share_a_workspace_in_turn():
    """Two captured steps over one workspace, replayed one after the other, with eager work between."""
    say("graphs over one workspace")
    M, H, I = 100, 2048, 128
    sets = [_ff_data(i, M, H, I, torch.bfloat16) for i in range(2)]
    gate_up = [cq.Fp8Weight(*cq.cubic_quant_fp8(s[1], block_rows=128)) for s in sets]
    n = max(cq.cubic_gated_ff_workspace_bytes(M, H, I), cq.cubic_gated_ff_backward_workspace_bytes(M, H, I), cq.cubic_gated_ff_fp8_workspace_bytes(M, H, I), 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def run(i, space):
        x, w, dh = sets[i]
        h, pre = cq.cubic_gated_ff(x, w, save_pre=True, workspace=space)
        return (h, *cq.cubic_gated_ff_backward(dh, x, w, pre, workspace=space), cq.cubic_gated_ff_fp8(x, gate_up[i], workspace=space))

    ref = [run(i, None) for i in range(2)]
    run(0, ws)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(run(i, ws))
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        eager = run(1 - i, None)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(outs[i], ref[i]))
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(eager, ref[1 - i]))


@pytest.mark.parametrize("M", [3, 80])
def test_one_tensor_twice(M):
    """Inputs may be one tensor: the gradient of h is x itself, and so is half of the weight."""
    say(f"one tensor twice M={M}")
    x, w, _ = _ff_data(M, M, 64, 64, torch.bfloat16)
    h, pre = cq.cubic_gated_ff(x, w, save_pre=True)
    dx, dw = cq.cubic_gated_ff_backward(x, x, w, pre)
    _check_grads(dx, dw, x, x, w, pre, "silu", torch.bfloat16)


def test_views_with_offsets():
    """Rows of larger tensors (16-byte offsets), and offsets that are not: refused."""
    say("views")
    x, w, dh = _ff_data(1, 40, 72, 24, torch.bfloat16)
    big = torch.empty(40 * 72 + 8, dtype=torch.bfloat16, device=DEV)
    v = big[8:].view(40, 72)
    v.copy_(x)
    assert torch.equal(bits(cq.cubic_gated_ff(v, w)), bits(cq.cubic_gated_ff(x, w)))
    off = torch.empty(40 * 72 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(40, 72)
    with pytest.raises(cq.CubicError):
        cq.cubic_gated_ff(off, w)
