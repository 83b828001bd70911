"""GPU parity of the gated feed-forward block and its backward pass against the oracle.

Tolerances (half: half a step of the type relative to the value, 2^-8 in bf16, 2^-11 in fp16; subnormal fp16
values 2^-25 absolute). pre: fp32 sums of exact products, e = (H + 8) 2^-24 S with S the sum of the terms'
magnitudes. h: e carried through |act'| <= 1.13 and |u|, |act|; the activation itself within 2^-18 of |g|
(exp's argument is rounded: |g| 2^-24 of it, up to |g| = 90 before exp leaves fp32); half a step. Gradients,
from the pre that the forward gave: each of dg, du off by half a step and by 2^-18 of |dh| (1 + |g|) max(|u|, 1)
for the slope, carried through the product's magnitudes; fp32 sums; half a step."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu
NAN = float("nan")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
F = lambda t: t.double().cpu().numpy()  # noqa: E731


def _guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), NAN, dtype=dtype, device=DEV)
    return buf[:n].view(shape), buf[n:]


def _data(seed, M, H, I, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((M, H), generator=g, device=DEV).to(dtype)
    w = (1.5 * torch.randn((2 * I, H), generator=g, device=DEV) / H ** 0.5).to(dtype)
    dh = torch.randn((M, I), generator=g, device=DEV).to(dtype)
    return x, w, dh


def _check_h(h, pre, x, w, act, dtype, extra=0.0):
    xd, wd = F(x), F(w)
    href, pref = oracle.gated_ff(xd, wd, act)
    e = (x.shape[1] + 8) * 2.0 ** -24 * (np.abs(xd) @ np.abs(wd).T) + extra
    if pre is not None:
        assert (np.abs(F(pre) - pref) <= e).all()
    I = h.shape[1]
    g, u = pref[:, :I], pref[:, I:]
    a = np.abs(oracle.act_and_slope(g, act)[0])
    tol = 1.13 * e[:, :I] * (np.abs(u) + e[:, I:]) + a * e[:, I:] + 2.0 ** -18 * np.abs(g * u)
    tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(href) + TINY[dtype]
    err = np.abs(F(h) - href)
    assert (err <= tol).all(), (err / tol).max()


def _check_grads(dx, dw, dh, x, w, pre, act, dtype):
    dhd, xd, wd, pd = F(dh), F(x), F(w), F(pre)
    dxr, dwr, dpre = oracle.gated_ff_backward(dhd, xd, wd, pd, act)
    M, I = dhd.shape
    g, u = pd[:, :I], pd[:, I:]
    one = 2.0 ** -18 * np.abs(dhd) * (1 + np.abs(g)) * np.maximum(np.abs(u), 1)
    de = np.concatenate([one, one], axis=1) + (HALF[dtype] * (1 + 2.0 ** -10)) * np.abs(dpre) + TINY[dtype]
    da = np.abs(dpre) + de
    if dx is not None:
        tol = de @ np.abs(wd) + (2 * I + 8) * 2.0 ** -24 * (da @ np.abs(wd))
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dxr) + TINY[dtype]
        assert (np.abs(F(dx) - dxr) <= tol).all(), (np.abs(F(dx) - dxr) / tol).max()
    if dw is not None:
        tol = de.T @ np.abs(xd) + (M + 8) * 2.0 ** -24 * (da.T @ np.abs(xd))
        tol = tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(dwr) + TINY[dtype]
        assert (np.abs(F(dw) - dwr) <= tol).all(), (np.abs(F(dw) - dwr) / tol).max()
        # roundings of single terms meet at random: no more than 1.5 times the result's own in the 2-norm, and a
        # part in a thousand for what the worst case above allows the sums
        for got, ref in ((dx, dxr), (dw, dwr)):
            if got is not None and ref.size > 4096:
                assert np.linalg.norm(F(got) - ref) <= (1.5 * HALF[dtype] / 3 ** 0.5 + 1e-5) * np.linalg.norm(ref)


SHAPES = [(1, 8, 8), (1, 512, 256), (2, 1000, 24), (7, 264, 520), (16, 2048, 128), (17, 40, 1000), (33, 520, 264), (45, 1000, 520),
          (64, 4104, 72), (65, 8, 136), (100, 1544, 680), (128, 128, 128), (200, 72, 2056), (257, 520, 328), (777, 136, 200), (1030, 264, 96)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,I", SHAPES)
def test_forward(M, H, I, act, dtype):
    say(f"gated_ff M={M} H={H} I={I} {act} {dtype}")
    x, w, _ = _data(M + H, M, H, I, dtype)
    h, guard = _guarded((M, I), dtype)
    pre, guard_p = _guarded((M, 2 * I), torch.float32)
    cq.cubic_gated_ff(x, w, act=act, out=h, pre=pre)
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_p).all())
    _check_h(h, pre, x, w, act, dtype)
    alone = cq.cubic_gated_ff(x, w, act=act)          # without pre: the same values
    assert torch.equal(alone.view(torch.int16), h.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,I", SHAPES)
def test_backward(M, H, I, act, dtype):
    say(f"gated_ff_backward M={M} H={H} I={I} {act} {dtype}")
    x, w, dh = _data(M + I, M, H, I, dtype)
    _, pre = cq.cubic_gated_ff(x, w, act=act, save_pre=True)
    dx, guard = _guarded((M, H), dtype)
    dw, guard_w = _guarded((2 * I, H), dtype)
    cq.cubic_gated_ff_backward(dh, x, w, pre, act=act, dx=dx, dw=dw)
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_w).all())
    _check_grads(dx, dw, dh, x, w, pre, act, dtype)
    for need_dx, need_dw in ((True, False), (False, True)):
        a, b = cq.cubic_gated_ff_backward(dh, x, w, pre, act=act, need_dx=need_dx, need_dw=need_dw)
        assert (a is None) == (not need_dx) and (b is None) == (not need_dw)
        got, ref = (a, dx) if need_dx else (b, dw)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """The directional derivative of sum(dh * h) from differences of the float64 formula, in random
    directions: off by the gradients' own roundings, which meet at random (five of their standard errors)."""
    say(f"gated_ff differences {act}")
    M, H, I = 40, 264, 136
    x, w, dh = _data(3, M, H, I, torch.float16)
    _, pre = cq.cubic_gated_ff(x, w, act=act, save_pre=True)
    dx, dw = (F(t) for t in cq.cubic_gated_ff_backward(dh, x, w, pre, act=act))
    xd, wd, dhd = F(x), F(w), F(dh)
    rng = np.random.default_rng(5)
    for _ in range(4):
        vx, vw = rng.normal(size=xd.shape), rng.normal(size=wd.shape)
        e = 1e-6
        loss = lambda s: float((oracle.gated_ff(xd + s * vx, wd + s * vw, act)[0] * dhd).sum())
        d = (loss(e) - loss(-e)) / (2 * e)
        rms = 2.0 ** -11 * 1.5 * np.sqrt(((dx * vx) ** 2).sum() + ((dw * vw) ** 2).sum())
        assert abs(d - ((dx * vx).sum() + (dw * vw).sum())) <= 5 * rms + 1e-6 * (np.abs(dx * vx).sum() + np.abs(dw * vw).sum())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_far_values(act):
    """Gates far out in both tails, zeros, and products that leave the type: x is a row of ones, so that
    gates and ups are sums of the weights."""
    say(f"gated_ff far values {act}")
    gates = torch.tensor([0.0, 1e-6, -1e-6, 3.0, -3.0, 12.0, -12.0, 30.0, -30.0, 88.0, -88.0, 100.0, -100.0, 1e4, -1e4, 2e4],
                         device=DEV, dtype=torch.bfloat16)
    w = torch.zeros((32, 16), dtype=torch.bfloat16, device=DEV)
    w[:16, 0], w[16:, 0] = gates, 1.0
    for M in (1, 70):
        x, dh = (torch.ones((M, n), dtype=torch.bfloat16, device=DEV) for n in (16, 16))
        h, pre = cq.cubic_gated_ff(x, w, act=act, save_pre=True)
        _check_h(h, pre, x, w, act, torch.bfloat16)
        dx, dw = cq.cubic_gated_ff_backward(dh, x, w, pre, act=act)
        _check_grads(dx, dw, dh, x, w, pre, act, torch.bfloat16)


@pytest.mark.parametrize("M", [1, 30, 90, 300])
def test_non_finite_stays_in_its_row(M):
    say(f"gated_ff non-finite M={M}")
    x, w, dh = _data(M, M, 264, 136, torch.bfloat16)
    clean, pre = cq.cubic_gated_ff(x, w, save_pre=True)
    cdx, _ = cq.cubic_gated_ff_backward(dh, x, w, pre)
    m, keep = M // 2, torch.arange(M, device=DEV) != M // 2
    for bad in (NAN, float("inf")):
        y = x.clone()
        y[m, 200] = bad
        h, p = cq.cubic_gated_ff(y, w, save_pre=True)
        assert not bool(torch.isfinite(p[m]).any())
        assert torch.equal(h[keep].view(torch.int16), clean[keep].view(torch.int16))
        d = dh.clone()
        d[m, 3] = bad
        dx, dw = cq.cubic_gated_ff_backward(d, x, w, pre)
        assert not bool(torch.isfinite(dx[m]).any()) and not bool(torch.isfinite(dw[3]).any()) and not bool(torch.isfinite(dw[136 + 3]).any())
        assert torch.equal(dx[keep].view(torch.int16), cdx[keep].view(torch.int16)) and bool(torch.isfinite(dw[4:136]).all())


@pytest.mark.parametrize("M", [1, 50, 90, 400])
def test_replays_streams_and_repeats(M):
    """A captured training step replayed between eager ones, two streams at once with their own workspaces."""
    say(f"gated_ff graph and streams M={M}")
    H, I = 512, 256
    sets = [_data(M + i, M, H, I, torch.bfloat16) for i in range(2)]

    def step(x, w, dh, ws=(None, None)):
        h, pre = cq.cubic_gated_ff(x, w, save_pre=True, workspace=ws[0])
        return (h, *cq.cubic_gated_ff_backward(dh, x, w, pre, workspace=ws[1]))

    same = lambda a, b: all(torch.equal(s.view(torch.int16), t.view(torch.int16)) for s, t in zip(a, b))  # noqa: E731
    ref = [step(*s) for s in sets]
    sizes = (max(1, cq.cubic_gated_ff_workspace_bytes(M, H, I)), max(1, cq.cubic_gated_ff_backward_workspace_bytes(M, H, I)))
    ws = [tuple(torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes) for _ in range(2)]
    held = [t.clone() for t in sets[0]]
    step(*held, ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*held, ws[0])
    for i in (1, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        for t in ws[0]:
            t.fill_(0xAA)
        graph.replay()
        eager = step(*sets[1 - i])
        torch.cuda.synchronize()
        assert same(out, ref[i]) and same(eager, ref[1 - i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([step(*sets[i], ws[i]) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(same(o, ref[i]) for i in range(2) for o in got[i])


def test_empty():
    say("gated_ff empty")
    x, w, dh = _data(1, 4, 64, 32, torch.bfloat16)
    h, pre = cq.cubic_gated_ff(x[:0], w, save_pre=True)
    assert h.shape == (0, 32) and pre.shape == (0, 64)
    dw = torch.full((64, 64), NAN, dtype=torch.bfloat16, device=DEV)
    dx, dw = cq.cubic_gated_ff_backward(dh[:0], x[:0], w, pre, dw=dw)
    assert dx.shape == (0, 64) and not bool(dw.any())


def _quantised(x):
    q, s = oracle.quant_fp8(F(x))
    return oracle.e4m3_values(q) * np.repeat(s.astype(np.float64), 128, axis=1)[:, :q.shape[1]]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,I", [(1, 16, 128), (1, 7168, 256), (3, 400, 384), (4, 8208, 128), (16, 1040, 256), (45, 528, 128), (65, 2048, 128),
                                   (130, 272, 512), (300, 1040, 384), (513, 144, 128)])
def test_fp8_block(M, H, I, act, out):
    say(f"gated_ff_fp8 M={M} H={H} I={I} {act} {out}")
    x, w, _ = _data(M + H, M, H, I, torch.bfloat16)
    wq, ws = cq.cubic_quant_fp8(w, block_rows=128)
    h, guard = _guarded((M, I), out)
    cq.cubic_gated_ff_fp8(x, cq.Fp8Weight(wq, ws), act=act, out=h, out_dtype=out)
    assert bool(torch.isnan(guard).all())
    xd = _quantised(x)
    wd = oracle.e4m3_values(wq.view(torch.uint8).cpu().numpy())
    wd = wd * np.repeat(np.repeat(ws.double().cpu().numpy(), 128, axis=0)[:2 * I], 128, axis=1)[:, :H]
    # the 8-bit MFMA drops what lies below 2^-14 of the largest of up to 128 products and the running sum
    kb = -(-H // 128)
    top = lambda t: np.pad(np.abs(t), ((0, 0), (0, kb * 128 - H))).reshape(t.shape[0], kb, 128).max(2)
    extra = 2 * 128 * 2.0 ** -14 * (top(xd) @ top(wd).T) + 4 * kb * 2.0 ** -24 * (np.abs(xd) @ np.abs(wd).T)
    as_t = lambda t: torch.from_numpy(t)
    _check_h(h, None, as_t(xd), as_t(wd), act, out, extra=extra)
    ref = oracle.gated_ff(xd, wd, act)[0]
    if ref.size > 1000:
        assert np.linalg.norm(F(h) - ref) <= (HALF[out] / 3 ** 0.5 + 2.0 ** -11) * np.linalg.norm(ref)


@pytest.mark.parametrize("M", [1, 37, 150])
def test_shared_expert(M):
    """The operators as a layer uses them: a 16-bit block is trained for a step, its weights quantised, and
    the expert served in 8 bits: gated block, then the down projection. Each stage follows the oracle of
    what the one before it gave."""
    say(f"shared expert M={M}")
    H, I = 512, 256
    x, w, dh = _data(M, M, H, I, torch.bfloat16)
    h, pre = cq.cubic_gated_ff(x, w, save_pre=True)
    dx, dw = cq.cubic_gated_ff_backward(dh, x, w, pre)
    _check_h(h, pre, x, w, "silu", torch.bfloat16)
    _check_grads(dx, dw, dh, x, w, pre, "silu", torch.bfloat16)
    w = w - 0.01 * dw
    gate_up = cq.Fp8Weight(*cq.cubic_quant_fp8(w, block_rows=128))
    down = (torch.randn((H, I), device=DEV, generator=torch.Generator(device=DEV).manual_seed(9)) / I ** 0.5).to(torch.bfloat16)
    down = cq.Fp8Weight(*cq.cubic_quant_fp8(down, block_rows=128))
    h8 = cq.cubic_gated_ff_fp8(x, gate_up)
    y = cq.cubic_linear_fp8(h8, down, out_dtype=torch.float32)
    gq = gate_up.codes.view(torch.uint8).cpu().numpy()
    gw = oracle.e4m3_values(gq) * np.repeat(np.repeat(F(gate_up.scales), 128, axis=0), 128, axis=1)
    ref = oracle.gated_ff(_quantised(x), gw, "silu")[0]
    assert np.linalg.norm(F(h8) - ref) <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11) * np.linalg.norm(ref)
    q, s = oracle.quant_fp8(F(h8))
    yref, S = oracle.gemm_fp8(q, s, down.codes.view(torch.uint8).cpu().numpy(), down.scales.cpu().numpy())
    assert (np.abs(F(y) - yref) <= (I + 8) * 2.0 ** -24 * S).all()


def test_binding_refuses():
    say("gated_ff binding refusals")
    x, w, dh = _data(1, 4, 64, 32, torch.bfloat16)
    _, pre = cq.cubic_gated_ff(x, w, save_pre=True)
    for call in (lambda: cq.cubic_gated_ff(x, w[:63]), lambda: cq.cubic_gated_ff(x, w[:, :56].contiguous()),
                 lambda: cq.cubic_gated_ff(x.half(), w), lambda: cq.cubic_gated_ff(x, w, act="relu"),
                 lambda: cq.cubic_gated_ff(x[:, ::2], w), lambda: cq.cubic_gated_ff(x, w, out=torch.empty((4, 31), dtype=torch.bfloat16, device=DEV)),
                 lambda: cq.cubic_gated_ff_backward(dh, x, w, pre.bfloat16()), lambda: cq.cubic_gated_ff_backward(dh[:3], x, w, pre),
                 lambda: cq.cubic_gated_ff_backward(dh.half(), x, w, pre)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(cq.CubicError):
        cq.cubic_gated_ff(x[:, :60].contiguous(), w[:, :60].contiguous())
