"""GPU parity of the int8 product (cubic_gemm_w8a8, cubic_linear_w8a8) against the oracle.

Tolerance: the dot product is exact; its conversion to fp32 and the two products round once each
(3 * 2^-24 relative to the product). With a bias the last product and the sum are one fused operation:
2 * 2^-24 of the product and 2^-24 of the result. A bf16 output is the fp32 one rounded, bit for bit."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _data(seed, M, N, K, bias, low=-128):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xq = torch.randint(low, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    wq = torch.randint(low, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sx = torch.exp(torch.randn((M,), generator=g, device=DEV) - 4)
    sw = torch.exp(torch.randn((N,), generator=g, device=DEV) - 4)
    b = 50 * torch.randn((N,), generator=g, device=DEV) if bias else None
    return xq, sx, cq.Int8Weight(wq, sw), b


def _np(*ts):
    return [None if t is None else t.cpu().numpy() for t in ts]


def _check(xq, sx, w, b, out_dtype=torch.float32):
    M, N = xq.shape[0], w.codes.shape[0]
    guard = torch.full((M * N + 256,), NAN, device=DEV)
    y = cq.cubic_gemm_w8a8(xq, sx, w, bias=b, out=guard[:M * N].view(M, N))
    assert bool(torch.isnan(guard[M * N:]).all())
    prod = oracle.gemm_w8a8(*_np(xq, sx, w.codes, w.scales))
    ref = prod if b is None else prod + b.cpu().numpy().astype(np.float64)[None, :]
    tol = 3 * 2.0 ** -24 * np.abs(prod) + (0 if b is None else 2.0 ** -24 * np.abs(ref))
    assert (np.abs(y.cpu().numpy().astype(np.float64) - ref) <= tol * (1 + 1e-6)).all()
    yb = cq.cubic_gemm_w8a8(xq, sx, w, bias=b, out_dtype=torch.bfloat16)
    assert torch.equal(yb.view(torch.int16), y.to(torch.bfloat16).view(torch.int16))
    return y


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 8), (16, 64), (37, 72), (300, 1000), (1003, 1928), (5000, 264), (40, 4104),
                                 (9000, 16)])
def test_rows_kernel(M, N, K):
    say(f"w8a8 rows M={M} N={N} K={K}")
    _check(*_data(M + N, M, N, K, bias=bool(M & 1)))


@pytest.mark.parametrize("M,N,K", [(65, 1, 8), (65, 64, 64), (128, 129, 72), (100, 4097, 136), (257, 300, 1000),
                                   (192, 1003, 1928), (513, 1030, 264), (1000, 2050, 48), (300, 6000, 200),
                                   (2049, 513, 328), (4096, 1537, 64), (1025, 3073, 24), (389, 28670, 136),
                                   (517, 12285, 72), (515, 14330, 200)])
def test_tile_kernel(M, N, K):
    say(f"w8a8 tiles M={M} N={N} K={K}")
    _check(*_data(M + N, M, N, K, bias=bool(N & 1)))


@pytest.mark.parametrize("M,N,K", [(3, 40, 131064), (70, 70, 131064), (64, 33, 20008)])
def test_long_sums(M, N, K):
    """The largest K, with rows whose int32 sums come close to 2^31."""
    say(f"w8a8 long K M={M} N={N} K={K}")
    xq, sx, w, b = _data(3, M, N, K, True)
    xq[0] = -128
    w.codes[0] = -128
    y = _check(xq, sx, w, b)
    ref = 16384.0 * K * float(sx[0]) * float(w.scales[0]) + float(b[0])
    assert abs(float(y[0, 0]) - ref) <= 4 * 2.0 ** -24 * abs(ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 500, 4096), (2, 77, 1928), (3, 1003, 72), (4, 64, 8192), (4, 30, 8), (5, 77, 200),
                                   (1, 50, 8200), (40, 100, 520), (200, 333, 264)])
def test_linear_equals_quantiser_then_product(M, N, K, dtype):
    say(f"w8a8 linear M={M} N={N} K={K} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn((M, K), generator=g, device=DEV)
    x[0, 0] = 31.0
    if M > 1:
        x[1] = 0                                      # a zero row: scale 0
    if M > 2:
        x[2] *= 1e-38 if dtype == torch.bfloat16 else 1e-6
    x = x.to(dtype)
    _, _, w, b = _data(K, M, N, K, True)
    xq, sx = (torch.from_numpy(v).to(DEV) for v in oracle.quant_w8a8(x.float().cpu().numpy()))
    near = cq.act_quant_int8_per_token(x)[1]          # divides instead: the last bit may differ
    assert bool(((near - sx).abs() <= 2.0 ** -23 * sx).all())
    for bias in (b, None):
        for od in (torch.float32, torch.bfloat16):
            want = cq.cubic_gemm_w8a8(xq, sx, w, bias=bias, out_dtype=od)
            got = cq.cubic_linear_w8a8(x, w, bias=bias, out_dtype=od)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    _check(xq, sx, w, b)


@pytest.mark.parametrize("M", [3, 700])
def test_linear_codes_at_halves(M):
    """Rows whose values lie at exact halves of the scale's steps (x = amax (2 n + 1) / 254): the codes
    follow the reciprocal rule and equal those of torch's quotients on the device."""
    say(f"w8a8 linear at halves M={M}")
    g = torch.Generator(device=DEV).manual_seed(M)
    K, N = 264, 40
    amax = (torch.randint(128, 256, (M, 1), generator=g, device=DEV) * 2.0 ** torch.randint(-9, 9, (M, 1), generator=g, device=DEV))
    x = (amax * (2 * torch.randint(-64, 64, (M, K), generator=g, device=DEV) + 1) / 254).to(torch.bfloat16)
    x[:, 0] = amax[:, 0].to(torch.bfloat16)
    x[:, 1] = (amax[:, 0] / 2).to(torch.bfloat16)
    xq, sx = (torch.from_numpy(v).to(DEV) for v in oracle.quant_w8a8(x.float().cpu().numpy()))
    ts = x.float().abs().amax(dim=1) / 127.0
    assert torch.equal(ts, sx) and torch.equal(torch.round(x.float() / ts[:, None]).to(torch.int8), xq)
    _, _, w, b = _data(M, M, N, K, True)
    assert torch.equal(cq.cubic_linear_w8a8(x, w, bias=b), cq.cubic_gemm_w8a8(xq, sx, w, bias=b))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("M,K", [(1, 64), (4, 4104), (6, 1928), (70, 136), (3, 8200), (5, 20000)])
def test_linear_non_finite_rows(M, K, bad):
    """A non-finite value makes its row non-finite, and no other row changes."""
    say(f"w8a8 linear non-finite M={M} K={K} {bad}")
    g = torch.Generator(device=DEV).manual_seed(K)
    _, _, w, b = _data(K, M, 50, K, True)
    x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    want = cq.cubic_linear_w8a8(x, w, bias=b)
    for dtype in (torch.bfloat16, torch.float16):
        for row, col in ((0, 0), (M - 1, K - 1), (M // 2, K // 2 + 3)):
            z = x.clone()
            z[row, col] = bad
            for od in (torch.float32, torch.bfloat16):
                y = cq.cubic_linear_w8a8(z.to(dtype), w, bias=b, out_dtype=od)
                assert not bool(y[row].isfinite().any())
                others = [m for m in range(M) if m != row]
                if dtype == torch.bfloat16 and od == torch.float32:
                    assert torch.equal(y[others], want[others])
                else:
                    assert bool(y[others].isfinite().all())


def test_large_shapes_sampled():
    """Full-size projections, checked on sampled rows and columns."""
    for M, N, K in ((1, 6144, 7168), (64, 7168, 7168), (96, 6144, 2048), (4096, 6144, 7168)):
        say(f"w8a8 large M={M} N={N} K={K}")
        xq, sx, w, b = _data(9, M, N, K, True)
        y = cq.cubic_gemm_w8a8(xq, sx, w, bias=b)
        rows = torch.unique(torch.tensor([0, M // 2, M - 1, min(M - 1, 255), min(M - 1, 256)], device=DEV))
        I = (xq[rows].double() @ w.codes.double().t())
        prod = I * w.scales.double() * sx[rows].double()[:, None]
        ref = prod + b.double()
        tol = 3 * 2.0 ** -24 * prod.abs() + 2.0 ** -24 * ref.abs()
        assert bool(((y[rows].double() - ref).abs() <= tol * (1 + 1e-6)).all())
        cols = torch.tensor([0, N - 1, N // 3], device=DEV)
        I = (xq.double() @ w.codes[cols].double().t())
        ref = I * w.scales[cols].double() * sx.double()[:, None] + b[cols].double()
        assert bool(((y[:, cols].double() - ref).abs() <= 4 * 2.0 ** -24 * (I * w.scales[cols].double() * sx.double()[:, None]).abs() + 2.0 ** -23 * ref.abs()).all())


def test_non_finite_scales_stay_in_their_rows():
    say("w8a8 non-finite scales")
    for M in (3, 80):
        xq, sx, w, b = _data(4, M, 50, 64, True)
        sx[1], sx[2] = NAN, float("inf")
        y = cq.cubic_gemm_w8a8(xq, sx, w, bias=b)
        assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).any())
        assert bool(torch.isfinite(y[0]).all()) and bool(torch.isfinite(y[3:]).all())


def test_weight_quantised_by_the_same_rule_and_shared_expert():
    """A run of the operators together: a dense weight quantised by its rows, a shared expert in W8A8
    beside the routed experts' router, in a captured graph replayed on new inputs."""
    say("w8a8 shared expert in a graph")
    g = torch.Generator(device=DEV).manual_seed(2)
    H, I, T = 512, 264, 6
    up = cq.Int8Weight(*cq.act_quant_int8_per_token(torch.randn((2 * I, H), generator=g, device=DEV).to(torch.bfloat16)))
    down = cq.Int8Weight(*cq.act_quant_int8_per_token(torch.randn((H, I), generator=g, device=DEV).to(torch.bfloat16)))
    gate = cq.Int8Weight(*cq.act_quant_int8_per_token(torch.randn((20, H), generator=g, device=DEV).to(torch.bfloat16)))

    def block(x):
        logits = cq.cubic_linear_w8a8(x, gate)
        ids, wts = cq.cubic_moe_topk(logits, 4, score="sigmoid")
        gu = cq.cubic_linear_w8a8(x, up)
        h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(torch.bfloat16)
        return ids, wts, cq.cubic_linear_w8a8(h, down, out_dtype=torch.bfloat16)

    xs = [torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]
    want = [[t.clone() for t in block(x)] for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    # against float64 on the quantised weights
    xq, sx = (torch.from_numpy(v).to(DEV) for v in oracle.quant_w8a8(xs[0].float().cpu().numpy()))
    gu = oracle.gemm_w8a8(*_np(xq, sx, up.codes, up.scales))
    h = gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]
    dense = down.codes.cpu().numpy().astype(np.float64) * down.scales.cpu().numpy().astype(np.float64)[:, None]
    y = want[0][2].float().cpu().numpy()
    # h: bf16 and per-row int8 (half a step of amax / 127 a value); y: bf16
    step = np.abs(h).max(axis=1, keepdims=True) / 254 + np.abs(h) * 2.0 ** -8
    tol = step @ np.abs(dense).T + 2.0 ** -7 * np.abs(h @ dense.T) + 1e-3
    assert (np.abs(y - h @ dense.T) <= tol).all()


def test_binding_refusals():
    xq, sx, w, b = _data(1, 3, 10, 64, True)
    with pytest.raises(TypeError):
        cq.cubic_gemm_w8a8(xq.float(), sx, w)
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq[:, :32].contiguous(), sx, w)
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq, sx[:2], w)
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq, sx, w, bias=b[:9])
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq, sx, cq.Int8Weight(w.codes, w.scales[:9]))
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq, sx, w, out=torch.empty((3, 11), device=DEV))
    with pytest.raises(ValueError):
        cq.cubic_gemm_w8a8(xq.t(), sx, w)
    with pytest.raises(TypeError):
        cq.cubic_linear_w8a8(xq.float(), w)
    y = cq.cubic_gemm_w8a8(xq[:0], sx[:0], w)
    assert y.shape == (0, 10)
