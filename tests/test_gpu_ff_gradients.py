"""Gradients of the gated feed-forward block where dg and du leave the range of fp16 while dx and dw do not, and the
gradients' 2-norm, each by itself. The references take the forward's pre in float64.

Tolerances. dg, du: the gate within 2^-18 |g| of its value and 2^-18 (1 + |g|) of its slope, half a step's rounding (1 + 2^-10 of
it), in fp16 2^-39 of the largest magnitude of the row (for dx) or the column (for dw) where that is more. Sums in
fp32 of n terms (n + 8) 2^-24 of their magnitudes; half a step of the type and its smallest step. In the
2-norm, where roundings of terms meet at random: the exact result's own rounding and one as large (1.42 times)."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say
from tests.test_gpu_gated_ff import F, HALF, TINY, _data, _guarded

pytestmark = pytest.mark.gpu
ACT = {torch.bfloat16: "silu", torch.float16: "gelu_tanh"}
bits = lambda t: t.view(torch.int16)  # noqa: E731


def _check(dx, dw, dh, x, w, pre, act, dtype):
    dhd, xd, wd, pd = F(dh), F(x), F(w), F(pre)
    M, I = dhd.shape
    g, u = pd[:, :I], pd[:, I:]
    dxr, dwr, dpre = oracle.gated_ff_backward(dhd, xd, wd, pd, act)
    gate = np.concatenate([2.0 ** -18 * np.abs(dhd * u) * (1 + np.abs(g)), 2.0 ** -18 * np.abs(dhd * g)], axis=1)
    a = np.abs(dpre)
    one = (gate + HALF[dtype] * a) * (1 + 2.0 ** -10) + (TINY[dtype] if dtype == torch.bfloat16 else 0.0)
    far = 0.0 if dtype == torch.bfloat16 else 2.0 ** -39
    if dx is not None:
        tol = (one + far * a.max(1, keepdims=True)) @ np.abs(wd) + (2 * I + 8) * 2.0 ** -24 * ((a + one) @ np.abs(wd))
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dxr) + TINY[dtype]
        assert (np.abs(F(dx) - dxr) <= tol).all(), (np.abs(F(dx) - dxr) / tol).max()
    if dw is not None:
        tol = (one + far * a.max(0, keepdims=True)).T @ np.abs(xd) + (M + 8) * 2.0 ** -24 * ((a + one).T @ np.abs(xd))
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dwr) + TINY[dtype]
        assert (np.abs(F(dw) - dwr) <= tol).all(), (np.abs(F(dw) - dwr) / tol).max()
    return dxr, dwr


# each tile shape, whole and in slices, ragged ends of both contractions, few rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(1, 4104, 520), (9, 1000, 264), (64, 1544, 680), (200, 512, 256), (777, 1544, 680), (515, 4104, 520), (2500, 2056, 1544),
                                   (2051, 4104, 1032), (3000, 136, 136), (300, 2056, 2056), (1030, 136, 2056)])
def test_two_norm(M, H, I, dtype):
    say(f"gated_ff_backward 2-norm M={M} H={H} I={I} {dtype}")
    x, w, dh = _data(M + I, M, H, I, dtype)
    pre = torch.randn((M, 2 * I), generator=torch.Generator(device=DEV).manual_seed(H), device=DEV)
    dx, guard = _guarded((M, H), dtype)
    dw, guard_w = _guarded((2 * I, H), dtype)
    need = cq.cubic_gated_ff_backward_workspace_bytes(M, H, I)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], dx=dx, dw=dw, workspace=ws[:need])
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_w).all()) and bool((ws[need:] == 0xFF).all())
    dxr, dwr = _check(dx, dw, dh, x, w, pre, ACT[dtype], dtype)
    for got, ref in ((dx, dxr), (dw, dwr)):           # each of them, whether the other one is there or not
        own = np.linalg.norm(F(torch.from_numpy(ref).to(dtype)) - ref)
        assert np.linalg.norm(F(got) - ref) <= 1.5 * own
    one, _ = cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], need_dw=False)
    _, two = cq.cubic_gated_ff_backward(dh, x, w, pre, act=ACT[dtype], need_dx=False)
    assert torch.equal(bits(one), bits(dx)) and torch.equal(bits(two), bits(dw))


# dg and du beyond 65504 (2^25), below 2^-25 (2^-34), and rows that are tiny throughout; dx and dw in range
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("lo,hi,size", [(-24, 15, 2.0 ** -14), (-24, -10, 2.0 ** 8), (-24, -23, 2.0 ** 8)])
@pytest.mark.parametrize("M,H,I", [(1, 264, 136), (40, 136, 72), (300, 520, 264), (4100, 72, 40)])
def test_fp16_gradients_outside_the_type(M, H, I, lo, hi, size, act):
    say(f"gated_ff_backward fp16 range M={M} H={H} I={I} 2^{lo}..2^{hi} {act}")
    g = torch.Generator(device=DEV).manual_seed(M)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rows = lo + torch.arange(M, device=DEV).remainder(hi - lo + 1)
    rows[0] = hi                                      # the largest row is there, whatever M
    cols = torch.arange(I, device=DEV).remainder(21) - 10
    dh = (r(M, I).sign() * torch.exp2(rows.float())[:, None]).half()
    pre = torch.cat([r(M, I), (1 + r(M, I).abs()) * torch.exp2(cols.float())], dim=1).contiguous()
    x, w = (r(M, H) * size / 4).half(), (r(2 * I, H) * size / 4).half()
    dx, dw = cq.cubic_gated_ff_backward(dh, x, w, pre, act=act)
    dxr, dwr = _check(dx, dw, dh, x, w, pre, act, torch.float16)
    assert np.isfinite(F(dx)).all() and np.isfinite(F(dw)).all() and np.abs(dxr).max() < 65504 and np.abs(dwr).max() < 65504


@pytest.mark.parametrize("M", [1, 50, 300])
def test_fp16_non_finite_stays_in_its_row_and_column(M):
    say(f"gated_ff_backward fp16 non-finite M={M}")
    H, I = 264, 136
    x, w, dh = _data(M, M, H, I, torch.float16)
    _, pre = cq.cubic_gated_ff(x, w, save_pre=True)
    cdx, cdw = cq.cubic_gated_ff_backward(dh, x, w, pre)
    m, rows = M // 2, torch.arange(M, device=DEV) != M // 2
    cols = torch.arange(2 * I, device=DEV) % I != 3
    for bad in (float("nan"), float("inf"), -float("inf")):
        d = dh.clone()
        d[m, 3] = bad
        dx, dw = cq.cubic_gated_ff_backward(d, x, w, pre)
        assert not bool(torch.isfinite(dx[m]).any()) and not bool(torch.isfinite(dw[~cols]).any())
        assert torch.equal(bits(dx[rows]), bits(cdx[rows])) and torch.equal(bits(dw[cols]), bits(cdw[cols]))


@pytest.mark.parametrize("M", [1, 90, 600])
def test_fp16_zeros_replays_and_streams(M):
    """Zero rows and columns; a captured pass over a workspace that others have written to, replayed between eager
    ones; two streams at once."""
    say(f"gated_ff_backward fp16 graph M={M}")
    H, I = 520, 264
    sets = []
    for i in range(2):
        x, w, dh = _data(M + i, M, H, I, torch.float16)
        dh = dh * 2.0 ** (-20 * i)
        dh[::3], dh[:, ::5] = 0, 0
        _, pre = cq.cubic_gated_ff(x, w, save_pre=True)
        sets.append((dh.contiguous(), x, w, pre))
    ref = [cq.cubic_gated_ff_backward(*s) for s in sets]
    for s, r in zip(sets, ref):
        _check(*r, *s, "silu", torch.float16)
        assert not bool(r[0][::3].any()) and not bool(r[1][:I:5].any()) and not bool(r[1][I::5].any())
    n = cq.cubic_gated_ff_backward_workspace_bytes(M, H, I)
    ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    held = [t.clone() for t in sets[0]]
    cq.cubic_gated_ff_backward(*held, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cq.cubic_gated_ff_backward(*held, workspace=ws[0])
    same = lambda a, b: all(torch.equal(bits(s), bits(t)) for s, t in zip(a, b))  # noqa: E731
    for i in (1, 0, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        ws[0].fill_(0xFF)
        graph.replay()
        eager = cq.cubic_gated_ff_backward(*sets[1 - i])
        torch.cuda.synchronize()
        assert same(out, ref[i]) and same(eager, ref[1 - i])
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([cq.cubic_gated_ff_backward(*sets[i], workspace=ws[i]) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(same(o, ref[i]) for i in range(2) for o in got[i])
