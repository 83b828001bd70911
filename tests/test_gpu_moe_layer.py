"""GPU parity of the router (cubic_moe_topk) and of the whole routed-expert layer for a few tokens
(cubic_moe_layer) against the float64 oracle.

Tolerances, from the arithmetic:
* ids are equal.
* weights: scores, sums and quotients in fp64, rounded to fp32 once: 2^-24 relative. (The softmax
  without a bias and without renormalisation is given 42 * 2^-24 here, as if its denominator were a
  sum in fp32; test_gpu_router_precision.py holds it to one rounding.)
* y in fp32, as a 2-norm: bars of 1e-3 to 5e-3, and 1e-2 per row for some wide codes. They are wide: they
  allow for sums off by 2^-16 and more, of which 2^-7 of the h values would round to a neighbour, and for
  levels in fp16. The two kernels' sums are exact and added up in fp32, and the levels of the composed
  path two bf16 halves; test_gpu_moe_layer_precision.py and test_gpu_moe_layer_composed.py hold them to
  the bounds that follow from that. A bf16 output adds half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, pack_fields, row_rel_err, say, x_bits

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _norm_err(y, ref):
    y, ref = np.asarray(y, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert np.array_equal(np.isfinite(y), np.isfinite(ref))
    d = np.linalg.norm(ref)
    return np.linalg.norm(y - ref) / d if d else float(np.abs(y).max())


# ------------------------------------------------------------------------------------------ the router


def _check_topk(logits, topk, score, bias=None, renorm=True, scale=1.0):
    ids = torch.full((logits.shape[0], topk), -7, dtype=torch.int32, device=DEV)
    w = torch.full((logits.shape[0], topk), NAN, device=DEV)
    cq.cubic_moe_topk(logits, topk, score=score, bias=bias, renormalize=renorm, scale=scale, topk_ids=ids,
                      topk_weights=w)
    ref_ids, ref_w = oracle.moe_topk(logits.double().cpu().numpy(), topk, score,
                                     None if bias is None else bias.cpu().numpy(), renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    w = w.cpu().numpy().astype(np.float64)
    tol = 42 * 2.0 ** -24 if score == "softmax" and bias is None and not renorm else 2.0 ** -24 * (1 + 1e-6)
    assert (np.abs(w - ref_w) <= tol * np.abs(ref_w) + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,topk", [(1, 896, 16), (5, 1, 1), (3, 64, 64), (7, 65, 64), (2, 8, 2), (33, 257, 9),
                                      (4, 1025, 10), (3, 2048, 64), (130, 1024, 1)])
def test_topk_against_oracle(T, E, topk, with_bias, score, dtype):
    say(f"topk T={T} E={E} topk={topk} {score} bias={with_bias} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(T * 10007 + E)
    logits = (1.5 * torch.randn((T, E), generator=g, device=DEV)).to(dtype)
    bias = 0.1 * torch.randn((E,), generator=g, device=DEV) if with_bias else None
    _check_topk(logits, topk, score, bias, renorm=True, scale=2.5)
    _check_topk(logits, topk, score, bias, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_topk_masks_ties_and_extremes(score, with_bias):
    say(f"topk masks and ties {score} bias={with_bias}")
    inf, big = float("inf"), torch.finfo(torch.float32).max
    T, E, topk = 12, 200, 6
    g = torch.Generator(device=DEV).manual_seed(3)
    L = torch.randn((T, E), generator=g, device=DEV)
    L[0] = -inf                                   # nothing left
    L[1] = NAN
    L[2, :] = -inf
    L[2, 150] = 0.5                               # one expert left
    L[3] = 1.25                                   # more ties than lanes
    L[4] = torch.where(torch.arange(E, device=DEV) % 2 == 0, 2.0, -inf)
    L[5, 7] = inf
    L[5, 11] = inf
    L[6] = -big                                   # the type's lowest value is a logit like others
    L[6, 60] = -0.9 * big
    L[7] = torch.where(torch.arange(E, device=DEV) % 3 == 0, 0.0, -0.0)
    L[8] = -120.0                                 # scores below fp32's range
    L[9, :100] = NAN
    L[10] = torch.linspace(-1e-6, 1e-6, E, device=DEV)
    L[11] = 40.0 + torch.linspace(-1, 1, E, device=DEV)       # sigmoids that round to one in fp32
    bias = None
    if with_bias:
        bias = torch.zeros((E,), device=DEV)
        bias[3], bias[60], bias[61], bias[62] = -inf, NAN, inf, inf
        bias[150:] = 1e-7 * torch.randn((50,), generator=g, device=DEV)
    _check_topk(L, topk, score, bias, renorm=True)
    _check_topk(L, topk, score, bias, renorm=False, scale=0.5)


def test_topk_close_biased_keys():
    """Keys closer together than fp32 resolves: more candidates than lanes, and fewer."""
    for E, spread in ((1500, 1e-9), (300, 1e-7), (40, 1e-10)):
        say(f"topk close keys E={E}")
        g = torch.Generator(device=DEV).manual_seed(E)
        L = spread * torch.randn((5, E), generator=g, device=DEV)
        _check_topk(L, 16, "sigmoid", torch.full((E,), 0.25, device=DEV))
        _check_topk(L, 16, "softmax", torch.full((E,), 0.25, device=DEV))


def test_topk_empty_and_views():
    ids, w = cq.cubic_moe_topk(torch.empty((0, 8), device=DEV), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    with pytest.raises(ValueError):
        cq.cubic_moe_topk(torch.zeros((8, 4), device=DEV).t(), 2)           # not contiguous
    with pytest.raises(cq.CubicError):
        cq.cubic_moe_topk(torch.zeros((2, 8), device=DEV), 9)
    with pytest.raises(cq.CubicError):
        cq.cubic_moe_topk(torch.zeros((9, 9), device=DEV)[1:], 2)           # 36 bytes off
    with pytest.raises(ValueError):
        cq.cubic_moe_topk(torch.zeros((2, 8), device=DEV), 2, score="tanh")
    with pytest.raises(ValueError):
        cq.cubic_moe_topk(torch.zeros((2, 8), device=DEV), 2, bias=torch.zeros((7,), device=DEV))


# ------------------------------------------------------------------------------------------- the layer


class Experts:
    """E back-to-back expert matrices [N][K] and their dense float64 weights."""

    def __init__(self, seed, E, N, K, bits, group, extra=0.0, wild=0.0):
        rng = np.random.default_rng(seed)
        km = (1 << (bits - 1)) - 1
        if bits == 2:
            codes = rng.choice([0, 0, 1, -1], size=(E, N, K)).astype(np.int8)
        else:
            codes = rng.integers(-km, km + 1, size=(E, N, K)).astype(np.int8)
        if extra:                                  # the field value that a symmetric quantiser never writes
            codes[rng.random(codes.shape) < extra] = -km - 1
        scales = (0.02 * np.exp(0.3 * rng.normal(size=(E, N, K // group)))).astype(np.float32)
        ab = np.stack([rng.uniform(0.6, 1.4, scales.shape), rng.uniform(-0.1, 0.2, scales.shape)], axis=-1)
        if wild:                                   # levels far from a line, and of either sign
            ab = rng.uniform(-wild, wild, ab.shape)
        shapes = ab.astype(np.float16).view(np.uint16)
        self.E, self.parts, self.bits, self.group = E, (codes, scales, shapes), bits, group
        packed = pack_fields(codes.reshape(E * N, K), bits)
        self.weight = cq.CubicWeight(torch.from_numpy(packed).to(DEV).reshape(-1),
                                     torch.from_numpy(scales).to(DEV).reshape(-1),
                                     torch.from_numpy(shapes.view(np.int16)).to(DEV).reshape(-1), N, K, bits, group)

    def dense(self, e):
        c, s, a = (v[e] for v in self.parts)
        return oracle.dequant(c, s, a, self.bits, self.group)


def _x(seed, T, H, outlier=20.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=DEV)
    x[:, torch.rand((H,), generator=g, device=DEV) < 0.01] *= outlier
    return x.to(torch.bfloat16)


def _logits(seed, T, E):
    return torch.randn((T, E), generator=torch.Generator(device=DEV).manual_seed(seed + 77), device=DEV)


def _run(x, logits, gu, dn, topk, out_dtype=torch.float32, poison=True, **kw):
    T, H = x.shape
    out = torch.full((T, H), NAN, dtype=out_dtype, device=DEV)
    n = cq.cubic_moe_layer_workspace_bytes(T, topk, gu.E, H, dn.weight.K)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    y, ids, w = cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, gu.E, topk, out=out, workspace=ws[:n],
                                   out_dtype=out_dtype, **kw)
    assert bool((ws[n:] == 0xFF).all())
    return y.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy()


def _reference(x, logits, gu, dn, topk, **kw):
    kw = dict(kw)
    bias = kw.pop("bias", None)
    return oracle.moe_layer(x_bits(x), logits.double().cpu().numpy(), topk, kw.pop("score", "softmax"), gu.dense,
                            dn.dense, None if bias is None else bias.cpu().numpy(), **kw)


@pytest.mark.parametrize("H,I,ug,dg", [(256, 128, 256, 128), (512, 256, 256, 256), (1024, 512, 512, 512),
                                       (384, 384, 128, 384), (1280, 640, 640, 128), (768, 1280, 384, 256),
                                       (2048, 128, 1024, 128)])
@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (1, 16, 16), (2, 5, 5), (3, 9, 4), (8, 6, 3), (5, 4, 1)])
def test_layer_two_bit(H, I, ug, dg, T, E, topk):
    say(f"layer W2 H={H} I={I} groups {ug}/{dg} T={T} E={E} topk={topk}")
    gu, dn = Experts(H + T, E, 2 * I, H, 2, ug), Experts(I + T, E, H, I, 2, dg)
    x, logits = _x(T, T, H), _logits(E, T, E)
    y, ids, w = _run(x, logits, gu, dn, topk, score="softmax")
    ref, rids, rw = _reference(x, logits, gu, dn, topk, score="softmax")
    assert np.array_equal(ids, rids) and np.allclose(w, rw, rtol=2.0 ** -23, atol=0)
    assert _norm_err(y, ref) <= 1e-3
    yb, _, _ = _run(x, logits, gu, dn, topk, torch.bfloat16, score="softmax")
    assert np.array_equal(yb, torch.from_numpy(y).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("T", [1, 3, 8])
def test_layer_unused_field(T):
    """Codes of -2 (level -q(2) s) in many tiles, or in a single place."""
    for extra in (0.1, 2e-6):
        say(f"layer W2 with codes of -2, T={T} share {extra}")
        gu, dn = Experts(5, 6, 512, 512, 2, 256, extra), Experts(6, 6, 512, 256, 2, 128, extra)
        x, logits = _x(7, T, 512), _logits(7, T, 6)
        y, _, _ = _run(x, logits, gu, dn, 3, score="sigmoid", scale=2.5)
        ref, _, _ = _reference(x, logits, gu, dn, 3, score="sigmoid", scale=2.5)
        assert _norm_err(y, ref) <= 1e-3


@pytest.mark.parametrize("bits,ug,dg", [(3, 128, 128), (4, 128, 256), (8, 256, 128)])
def test_layer_wide_codes(bits, ug, dg):
    say(f"layer bits={bits}")
    gu, dn = Experts(bits, 6, 512, 512, bits, ug), Experts(bits + 1, 6, 512, 256, bits, dg)
    for T in (1, 4):
        x, logits = _x(T, T, 512), _logits(T, T, 6)
        y, ids, _ = _run(x, logits, gu, dn, 3)
        ref, rids, _ = _reference(x, logits, gu, dn, 3)
        assert np.array_equal(ids, rids) and row_rel_err(y, ref) <= 1e-2
        yb, _, _ = _run(x, logits, gu, dn, 3, torch.bfloat16)
        assert np.array_equal(yb, torch.from_numpy(y).to(torch.bfloat16).float().numpy())


@pytest.mark.parametrize("bits", [3, 4])
@pytest.mark.parametrize("H,I,ug,dg", [(256, 128, 128, 128), (768, 640, 384, 640), (1152, 256, 128, 256),
                                       (2048, 512, 512, 128)])
def test_layer_wide_codes_in_two_kernels(bits, H, I, ug, dg):
    """3- and 4-bit codes, the field value -2^(B-1) among them, one to eight tokens. Sums are off by some
    2^-16, so that 2^-7 of the h values may round to a neighbour, up to 2^-7 off: a 2-norm error of
    2^-7 * 2^-3.5 = 7e-4 where h values are alike, and more where one h makes up much of a row (a single
    h of -5.86 among values below one that rounds the other way: 1.5e-3); the bar is 2e-3."""
    for T, E, topk in ((1, 5, 5), (3, 9, 2), (8, 6, 4)):
        say(f"layer bits={bits} H={H} I={I} groups {ug}/{dg} T={T}")
        gu, dn = Experts(bits + T, E, 2 * I, H, bits, ug, 0.01), Experts(T, E, H, I, bits, dg, 0.01)
        x, logits = _x(T, T, H), _logits(T, T, E)
        if T == 3:
            logits[1] = -float("inf")
        y, ids, w = _run(x, logits, gu, dn, topk, score="sigmoid")
        ref, rids, _ = _reference(x, logits, gu, dn, topk, score="sigmoid")
        assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 2e-3
        again, _, _ = _run(x, logits, gu, dn, topk, score="sigmoid")
        assert np.array_equal(y, again)


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_layer_levels_of_any_shape(bits):
    """a and b in -4 .. 4, so that a level's parts are up to 2^4 times itself and cancel: sums off by some
    2^-12, and 2^-3 of the h values round to a neighbour, up to 2^-7 off (2^-7 * 2^-1.5 = 2.8e-3); the bar
    is 5e-3."""
    gu, dn = Experts(1, 6, 512, 768, bits, 128, 0.02, 4.0), Experts(2, 6, 768, 256, bits, 128, 0.02, 4.0)
    for T in (1, 6):
        say(f"layer bits={bits} wild shapes T={T}")
        x, logits = _x(T, T, 768), _logits(T, T, 6)
        y, ids, _ = _run(x, logits, gu, dn, 3, score="sigmoid")
        ref, rids, _ = _reference(x, logits, gu, dn, 3, score="sigmoid")
        assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 5e-3


@pytest.mark.parametrize("ub,db", [(2, 4), (4, 2), (3, 2), (2, 3), (4, 3), (2, 6)])
def test_layer_mixed_widths(ub, db):
    say(f"layer bits {ub}/{db}")
    gu, dn = Experts(ub, 6, 512, 512, ub, 256), Experts(db, 6, 512, 256, db, 128)
    for T in (1, 5):
        x, logits = _x(T, T, 512), _logits(T, T, 6)
        y, ids, _ = _run(x, logits, gu, dn, 3)
        ref, rids, _ = _reference(x, logits, gu, dn, 3)
        assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 2e-3


@pytest.mark.parametrize("bits,T", [(2, 9), (2, 21), (2, 32), (2, 33), (2, 40), (2, 41), (2, 64), (2, 65), (3, 50),
                                     (4, 9), (4, 16), (4, 17), (4, 33), (4, 64), (4, 65)])
def test_layer_runs_of_tokens(bits, T):
    """More than eight tokens, with weights above 4 MB: runs of up to eight on the same buffers, then the
    composed path."""
    say(f"layer runs bits={bits} T={T}")
    H, I, E, topk = 1024, 512, 12, 3
    gu, dn = Experts(T, E, 2 * I, H, bits, 256), Experts(T + 1, E, H, I, bits, 256)
    x, logits = _x(T, T, H), _logits(T, T, E)
    logits[T // 2] = -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        y, ids, w = _run(x, logits.to(dtype), gu, dn, topk, score="sigmoid", scale=2.5)
        ref, rids, rw = _reference(x, logits.to(dtype), gu, dn, topk, score="sigmoid", scale=2.5)
        assert np.array_equal(ids, rids) and np.allclose(w, rw, rtol=2.0 ** -23, atol=0)
        assert _norm_err(y, ref) <= 2e-3


@pytest.mark.parametrize("T,E,topk", [(8, 70, 64), (2, 300, 20), (1, 1024, 16), (1, 1025, 16)])
def test_layer_many_experts(T, E, topk):
    """Routers of 4 and 16 experts a lane, 512 pairs, and more experts than the two kernels take."""
    say(f"layer E={E} topk={topk} T={T}")
    H, I = 256, 128
    gu, dn = Experts(1, E, 2 * I, H, 2, 256), Experts(2, E, H, I, 2, 128)
    x, logits = _x(T, T, H), _logits(T, T, E)
    y, ids, _ = _run(x, logits, gu, dn, topk)
    ref, rids, _ = _reference(x, logits, gu, dn, topk)
    assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 1e-3


@pytest.mark.parametrize("H,T", [(9216, 8), (10240, 8), (16384, 1), (20480, 4)])
def test_layer_long_rows(H, T):
    """Rows around and beyond what the two kernels hold in LDS; output rows in more than 256 blocks."""
    say(f"layer H={H} T={T}")
    I, E, topk = 256, 3, 2
    gu, dn = Experts(1, E, 2 * I, H, 2, 512), Experts(2, E, H, I, 2, 256)
    x, logits = _x(T, T, H), _logits(T, T, E)
    y, ids, _ = _run(x, logits, gu, dn, topk)
    ref, rids, _ = _reference(x, logits, gu, dn, topk)
    assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 1e-3


def test_layer_long_intermediate():
    """h rows longer than a wave's share of LDS: K parts in kernel 2."""
    for bits, I, T in ((2, 8192, 1), (2, 12800, 2), (4, 6144, 1)):
        say(f"layer bits={bits} I={I} T={T}")
        gu, dn = Experts(1, 2, 2 * I, 256, bits, 128), Experts(2, 2, 256, I, bits, 256)
        x, logits = _x(T, T, 256), _logits(T, T, 2)
        y, _, _ = _run(x, logits, gu, dn, 2)
        ref, _, _ = _reference(x, logits, gu, dn, 2)
        assert _norm_err(y, ref) <= 2e-3


def test_layer_mixed_widths_and_more_tokens():
    say("layer W3 gate_up, W2 down; then W2 with 9 and 40 tokens")
    gu, dn = Experts(1, 6, 512, 512, 3, 256), Experts(2, 6, 512, 256, 2, 256)
    x, logits = _x(4, 4, 512), _logits(4, 4, 6)
    assert row_rel_err(_run(x, logits, gu, dn, 3)[0], _reference(x, logits, gu, dn, 3)[0]) <= 1e-2
    gu = Experts(3, 6, 512, 512, 2, 256)
    for T in (9, 40):
        x, logits = _x(T, T, 512), _logits(T, T, 6)
        y, ids, _ = _run(x, logits, gu, dn, 3)
        ref, rids, _ = _reference(x, logits, gu, dn, 3)
        assert np.array_equal(ids, rids) and _norm_err(y, ref) <= 1e-3


def test_layer_equals_router_then_mlp():
    """A run of the operators as they are used: the router, the MLP step over its ids and weights, and
    the layer that does both; large expert shapes."""
    say("layer against topk + moe_mlp, H=7168 I=1536")
    H, I, E, topk = 7168, 1536, 6, 4
    gu, dn = Experts(11, E, 2 * I, H, 2, 512), Experts(12, E, H, I, 2, 512)
    for T in (1, 4, 8):
        x, logits = _x(T, T, H), _logits(T, T, E)
        bias = 0.1 * torch.randn((E,), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV)
        ids, w = cq.cubic_moe_topk(logits, topk, score="sigmoid", bias=bias, scale=2.5)
        step = cq.cubic_moe_mlp(x, ids, w, gu.weight, dn.weight, E).cpu().numpy()
        y, lids, lw = _run(x, logits, gu, dn, topk, score="sigmoid", bias=bias, scale=2.5)
        assert np.array_equal(lids, ids.cpu().numpy()) and np.array_equal(lw, w.cpu().numpy())
        assert _norm_err(y, step) <= 1e-3
        again, _, _ = _run(x, logits, gu, dn, topk, score="sigmoid", bias=bias, scale=2.5)
        assert np.array_equal(y, again)


def test_layer_masked_tokens_and_non_finite_rows():
    say("layer: masked rows, a NaN and an infinite activation")
    gu, dn = Experts(21, 6, 512, 512, 2, 256), Experts(22, 6, 512, 256, 2, 256)
    T = 6
    x, logits = _x(1, T, 512), _logits(1, T, 6)
    logits[1] = -float("inf")                       # no expert at all
    logits[2, 1:] = -float("inf")                   # one expert, two slots empty
    x[4, 100], x[5, 3] = NAN, float("inf")
    out = _run(x, logits, gu, dn, 3)[0]
    clean = x.clone()
    clean[4:] = 0
    ref, rids, _ = _reference(clean, logits, gu, dn, 3)
    assert not out[1].any() and np.isnan(out[4]).all() and not np.isfinite(out[5]).any()
    assert _norm_err(out[:4], ref[:4]) <= 1e-3
    assert (rids[1] == -1).all()
    logits[:] = -float("inf")
    y, ids, w = _run(x, logits, gu, dn, 3)
    assert not y.any() and (ids == -1).all() and not w.any()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e4, 1e12])
def test_layer_activation_range(scale):
    """Small and large activations, and channels 2^13 above the others that some rows do not read."""
    say(f"layer activations of size {scale}")
    gu, dn = Experts(31, 4, 512, 512, 2, 256), Experts(32, 4, 512, 256, 2, 256)
    for outlier in (1.0, 2.0 ** 13):
        g = torch.Generator(device=DEV).manual_seed(8)
        x = torch.randn((2, 512), generator=g, device=DEV)
        x[:, 5::64] *= outlier
        x = (x * scale).to(torch.bfloat16)
        logits = _logits(8, 2, 4)
        y, _, _ = _run(x, logits, gu, dn, 2)
        ref, _, _ = _reference(x, logits, gu, dn, 2)
        if scale == 1e-30:                          # h underflows to zero for the larger part
            assert np.abs(y - ref).max() <= 1e-30
        else:
            assert _norm_err(y, ref) <= 1e-3


def test_layer_streams_and_graph():
    """Side streams with a workspace each, and a captured layer replayed on new inputs between eager
    work."""
    say("layer on two streams and in a graph")
    gu, dn = Experts(41, 8, 1024, 512, 2, 256), Experts(42, 8, 512, 512, 2, 256)
    xs = [_x(s, 2, 512) for s in range(4)]
    ls = [_logits(s, 2, 8) for s in range(4)]
    want = [_run(x, l, gu, dn, 3)[0] for x, l in zip(xs, ls)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(cq.cubic_moe_layer(xs[i], ls[i], gu.weight, dn.weight, 8, 3, out_dtype=torch.float32)[0])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy(), w)
    x, l = xs[0].clone(), ls[0].clone()
    out = torch.empty((2, 512), device=DEV)
    ws = torch.empty(cq.cubic_moe_layer_workspace_bytes(2, 3, 8, 512, 512), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        cq.cubic_moe_layer(x, l, gu.weight, dn.weight, 8, 3, out=out, workspace=ws, out_dtype=torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cq.cubic_moe_layer(x, l, gu.weight, dn.weight, 8, 3, out=out, workspace=ws, out_dtype=torch.float32)
    for i in (1, 2, 3, 0, 2):
        x.copy_(xs[i])
        l.copy_(ls[i])
        out.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want[i])


def test_layer_binding_refusals():
    gu, dn = Experts(51, 4, 512, 512, 2, 256), Experts(52, 4, 512, 256, 2, 256)
    x, logits = _x(1, 2, 512), _logits(1, 2, 4)
    call = lambda x=x, logits=logits, E=4, topk=2, **kw: cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, E, topk,
                                                                            **kw)
    with pytest.raises(TypeError):
        call(x=x.float())
    with pytest.raises(ValueError):
        call(E=5)
    with pytest.raises(ValueError):
        call(logits=_logits(1, 3, 4))
    with pytest.raises(ValueError):                  # more experts than the weights hold
        call(logits=_logits(1, 2, 6), E=6)
    with pytest.raises(TypeError):
        call(out_dtype=torch.float16)
    with pytest.raises(ValueError):
        call(out=torch.empty((2, 256), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(cq.CubicError):
        call(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(cq.CubicError):
        call(topk=5)
    y, ids, w = call(x=x[:0], logits=logits[:0])
    assert y.shape == (0, 512) and ids.shape == (0, 2)
