"""GPU parity of the e4m3 quantiser and product against the oracle.

Tolerances. Quantiser: bit for bit. Product, fp32 out: products are exact, a block's sum and the sum over
blocks are fp32 in some order and each block's scale is rounded once, so |error| <= (K + 4 blocks) 2^-24 S
with S the sum of the terms' magnitudes. 16-bit out: half a step of the type (2^-8 or 2^-11 relative, 2^-25
where fp16 is subnormal) and, since such products may run on the 8-bit MFMA, which aligns up to 128 products
and the running sum to their largest and drops what lies below 2^-14 of it, 2 * 128 * 2^-14 of a block's largest
product a block, at the very most; in the 2-norm, where such errors meet at random, 2^-13."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _np(t):
    return None if t is None else (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).cpu().numpy()


def _guarded(shape, dtype):
    """(a view of this shape, what lies behind it): NaN everywhere."""
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), NAN, dtype=dtype, device=DEV)
    return buf[:n].view(shape), buf[n:]


def _acts(g, M, K, dtype=torch.bfloat16):
    x = torch.randn((M, K), generator=g, device=DEV)
    return torch.where(torch.rand((K,), generator=g, device=DEV) < 0.02, 20 * x, x).to(dtype)


def _data(seed, M, N, K, bias=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    xq, xs = cq.cubic_quant_fp8(_acts(g, M, K))
    w = (torch.randn((N, K), generator=g, device=DEV) * torch.exp(torch.randn((N, 1), generator=g, device=DEV)) / K ** 0.5)
    wq, ws = cq.cubic_quant_fp8(w.to(torch.bfloat16), block_rows=128)
    b = torch.randn((N,), generator=g, device=DEV) if bias else None
    return xq, xs, cq.Fp8Weight(wq, ws), b


def _check(y, xq, xs, w, b, out_dtype):
    K = xq.shape[1]
    ref, S = oracle.gemm_fp8(_np(xq), _np(xs), _np(w.codes), _np(w.scales), _np(b))
    kb = -(-K // 128)
    tol = (K + 4 * kb) * 2.0 ** -24 * S + HALF[out_dtype] * np.abs(ref) * 1.001 + (2.0 ** -25 if out_dtype == torch.float16 else 0)
    err = np.abs(y.double().cpu().numpy() - ref)
    if out_dtype != torch.float32:
        pad = lambda q: np.pad(np.abs(oracle.e4m3_values(_np(q))), ((0, 0), (0, kb * 128 - K))).reshape(q.shape[0], kb, 128).max(2)
        px = pad(xq) * _np(xs).astype(np.float64)
        pw = pad(w.codes) * np.repeat(_np(w.scales).astype(np.float64), 128, axis=0)[:w.codes.shape[0]]
        tol = tol + 2 * 128 * 2.0 ** -14 * (px @ pw.T)
        assert np.linalg.norm(err) <= (HALF[out_dtype] / 3 ** 0.5 + 2.0 ** -13) * np.linalg.norm(ref) + 1e-30
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (128, 144), (130, 272), (257, 1040), (5, 7168)])
def test_quantiser(M, K, rows, dtype):
    say(f"quant_fp8 M={M} K={K} rows={rows} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = _acts(g, M, K, dtype)
    x[0, :min(128, K)] = 0                            # with one row a scale of zero
    x[-1, -8:] = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -130
    if M > 2:
        x[1] = 65504.0 if dtype == torch.float16 else 3e38
    codes = torch.full((M * K + 64,), 0x55, dtype=torch.uint8, device=DEV)
    scales, guard = _guarded((-(-M // rows), -(-K // 128)), torch.float32)
    q, s = cq.cubic_quant_fp8(x, rows, xq=codes[:M * K].view(torch.float8_e4m3fn).view(M, K), scales=scales)
    qr, sr = oracle.quant_fp8(x.double().cpu().numpy(), rows)
    assert np.array_equal(_np(s), sr)
    assert np.array_equal(_np(q), qr) or np.array_equal(oracle.e4m3_values(_np(q)), oracle.e4m3_values(qr))
    assert bool((codes[M * K:] == 0x55).all()) and bool(torch.isnan(guard).all())


def test_quantiser_ties():
    """Quotients exactly halfway between codes: amax 448 gives a scale of one."""
    say("quant_fp8 ties")
    table = oracle.e4m3_values(np.arange(127, dtype=np.uint8))
    mids = (table[:-1] + table[1:]) / 2
    x = torch.zeros((1, 128), dtype=torch.float32, device=DEV)
    x[0, :126] = torch.from_numpy(mids).float()
    x[0, 126], x[0, 127] = 448.0, -448.0
    q, s = cq.cubic_quant_fp8(x.to(torch.bfloat16))   # five significant bits: exact in bf16
    assert float(s) == 1.0
    assert np.array_equal(_np(q), oracle.e4m3_round(x.double().cpu().numpy()))


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_quantiser_non_finite(bad, rows):
    say(f"quant_fp8 {bad} rows={rows}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = _acts(g, 200, 256)
    clean = cq.cubic_quant_fp8(x, rows)
    x[3, 130] = bad
    q, s = cq.cubic_quant_fp8(x, rows)
    at = 3 // rows
    assert not bool(torch.isfinite(s[at, 1])) and bool(torch.isnan(q[3, 130].float()))
    s[at, 1], q[at * rows:(at + 1) * rows, 128:] = clean[1][at, 1], clean[0][at * rows:(at + 1) * rows, 128:]
    assert torch.equal(s, clean[1]) and torch.equal(q.view(torch.uint8), clean[0].view(torch.uint8))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 16, 128), (1, 500, 1040), (2, 37, 144), (4, 300, 4112), (5, 129, 272), (16, 1003, 1936),
                                   (17, 260, 528), (33, 2050, 400), (37, 1003, 1936), (64, 520, 2048), (1, 6144, 7168), (3, 40, 9232)])
def test_few_rows(M, N, K, out):
    say(f"gemm_fp8 few rows M={M} N={N} K={K} {out}")
    xq, xs, w, b = _data(M + N, M, N, K, bias=bool(N & 1))
    y, guard = _guarded((M, N), out)
    cq.cubic_gemm_fp8(xq, xs, w, bias=b, out=y, out_dtype=out)
    assert bool(torch.isnan(guard).all())
    _check(y, xq, xs, w, b, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(65, 1, 16), (65, 64, 144), (100, 4097, 272), (128, 130, 128), (129, 257, 256), (200, 500, 1040),
                                   (257, 300, 1000 // 16 * 16), (300, 6000, 208), (513, 1030, 400), (700, 384, 7168), (1025, 2050, 48),
                                   (80, 7168, 2048)])
def test_many_rows(M, N, K, out):
    say(f"gemm_fp8 many rows M={M} N={N} K={K} {out}")
    xq, xs, w, b = _data(M + N, M, N, K, bias=bool(N & 1))
    y, guard = _guarded((M, N), out)
    cq.cubic_gemm_fp8(xq, xs, w, bias=b, out=y, out_dtype=out)
    assert bool(torch.isnan(guard).all())
    _check(y, xq, xs, w, b, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 40, 100, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear_equals_quantiser_and_product(M, dtype, out):
    say(f"linear_fp8 M={M} {dtype} {out}")
    g = torch.Generator(device=DEV).manual_seed(M)
    for N, K in ((300, 1040), (1003, 8208)):
        x = _acts(g, M, K, dtype)
        x[0, :128] = 0
        _, _, w, b = _data(M + 1, 1, N, K, bias=True)
        y = cq.cubic_linear_fp8(x, w, bias=b, out_dtype=out)
        xq, xs = cq.cubic_quant_fp8(x)
        _check(y, xq, xs, w, b, out)


@pytest.mark.parametrize("M", [1, 3, 20, 70, 300])
def test_non_finite_stays_in_its_row_and_columns(M):
    say(f"fp8 non-finite M={M}")
    g = torch.Generator(device=DEV).manual_seed(M)
    x = _acts(g, M, 528)
    _, _, w, _ = _data(5, 1, 270, 528)
    clean = cq.cubic_linear_fp8(x, w, out_dtype=torch.bfloat16)
    m = M // 2
    for bad in (NAN, float("inf")):
        y = x.clone()
        y[m, 500] = bad
        got = cq.cubic_linear_fp8(y, w, out_dtype=torch.bfloat16)
        assert not bool(torch.isfinite(got[m]).any())
        keep = torch.arange(M, device=DEV) != m
        assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    codes = w.codes.clone()
    codes.view(torch.uint8)[200, 17] = 0x7F           # one NaN weight: its column of y
    got = cq.cubic_linear_fp8(x, cq.Fp8Weight(codes, w.scales), out_dtype=torch.bfloat16)
    keep = torch.arange(270, device=DEV) != 200
    assert bool(torch.isnan(got[:, 200]).all())
    assert torch.equal(got[:, keep].view(torch.int16), clean[:, keep].view(torch.int16))


def test_cut_blocks_use_their_own_scales():
    """Large scales in the blocks cut at the edges: what lies behind N and K is not read into them."""
    say("fp8 cut blocks")
    for M in (1, 40, 90, 260):
        xq, xs, w, _ = _data(M, M, 140, 400)
        w.scales[1] *= 1e6
        w.scales[:, 3] *= 1e3
        xs[:, 3] *= 1e3
        _check(cq.cubic_gemm_fp8(xq, xs, w), xq, xs, w, None, torch.float32)


@pytest.mark.parametrize("M", [1, 4, 50, 90, 700])
def test_replays_streams_and_repeats(M):
    """A captured graph replayed between eager work, another stream, two calls at once with their own
    workspaces: every result equal bit for bit."""
    say(f"fp8 graph and streams M={M}")
    N, K = 520, 2048
    g = torch.Generator(device=DEV).manual_seed(M)
    xs_ = [_acts(g, M, K) for _ in range(3)]
    _, _, w, _ = _data(M, 1, N, K)
    ref = [cq.cubic_linear_fp8(x, w, out_dtype=torch.bfloat16) for x in xs_]
    need = max(1, cq.cubic_linear_fp8_workspace_bytes(M, N, K))
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    x, y = xs_[0].clone(), torch.empty_like(ref[0])
    cq.cubic_linear_fp8(x, w, out=y, workspace=ws[0], out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cq.cubic_linear_fp8(x, w, out=y, workspace=ws[0], out_dtype=torch.bfloat16)
    for i in (1, 2, 0, 1):
        x.copy_(xs_[i])
        ws[0].fill_(0xAA)
        graph.replay()
        eager = cq.cubic_linear_fp8(xs_[2], w, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), ref[i].view(torch.int16)) and torch.equal(eager.view(torch.int16), ref[2].view(torch.int16))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs.append([cq.cubic_linear_fp8(xs_[i], w, workspace=ws[i], out_dtype=torch.bfloat16) for _ in range(5)])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.view(torch.int16), ref[i].view(torch.int16)) for o in outs[i])


def test_empty():
    say("fp8 empty")
    _, _, w, _ = _data(1, 1, 40, 128)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    assert cq.cubic_linear_fp8(x, w).shape == (0, 40) and cq.cubic_quant_fp8(x)[1].shape == (0, 1)
    none = cq.Fp8Weight(w.codes[:0], w.scales[:0])
    assert cq.cubic_linear_fp8(torch.zeros((3, 128), dtype=torch.bfloat16, device=DEV), none).shape == (3, 0)


def test_binding_refuses():
    say("fp8 binding refusals")
    xq, xs, w, _ = _data(1, 4, 40, 256)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: cq.cubic_gemm_fp8(xq, xs[:, :1].contiguous(), w), lambda: cq.cubic_gemm_fp8(xq[:, :128].contiguous(), xs, w),
                 lambda: cq.cubic_linear_fp8(x.t().contiguous().t(), w), lambda: cq.cubic_linear_fp8(x[:, ::2], w),
                 lambda: cq.cubic_gemm_fp8(xq, xs, cq.Fp8Weight(w.codes, w.scales[:, :1].contiguous())),
                 lambda: cq.cubic_linear_fp8(x, w, out=torch.empty((4, 41), device=DEV)),
                 lambda: cq.cubic_linear_fp8(x, w, bias=torch.zeros(39, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(TypeError):
        cq.cubic_linear_fp8(x, w, out_dtype=torch.float64)
    with pytest.raises(cq.CubicError):
        cq.cubic_quant_fp8(x[:, :8].contiguous())
