"""Precision of the routed-expert layer's sums (cubic_moe_layer) for a few tokens: small activations
beside outliers that a row does not read, large products that cancel, and long sums of ordinary ones.

Bounds, from the arithmetic. A sum of n codes runs as exact integer sums of 128 or 256 products each,
which fp32 adds up: with S = sum |x_k| |level_k| (3 and 4 bits: the level as the sum of its three parts'
magnitudes) it is off by at most eps * S, eps = (3 n / 128 + 24) * 2^-24 (three fp32 additions a step for
the three parts, up to eight waves' sums, the parts' coefficients), and, as an activation is a multiple
of 2^-29 of its block's largest power of two, by 2^-30 * max |x| of 256 neighbours * sum |level|.
h = bf16(v): where v lies closer to a rounding border than g's and u's bounds carry it (and 2^-20 of v
for expf and its quotient), h may be either neighbour. y's bound adds those steps through the down
levels to its own sum's bound.
"""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, pack_fields, say, x_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


class Experts:
    """E matrices [N][K]: codes, scales, shapes (numpy), their weight, levels and parts' magnitudes."""

    def __init__(self, seed, E, N, K, bits, group):
        rng = np.random.default_rng(seed)
        km = (1 << (bits - 1)) - 1
        if bits == 2:
            self.codes = rng.choice([0, 0, 1, -1], size=(E, N, K)).astype(np.int8)
        else:
            self.codes = rng.integers(-km, km + 1, size=(E, N, K)).astype(np.int8)
        self.scales = (0.02 * np.exp(0.3 * rng.normal(size=(E, N, K // group)))).astype(np.float32)
        ab = np.stack([rng.uniform(0.6, 1.4, self.scales.shape), rng.uniform(-0.1, 0.2, self.scales.shape)], axis=-1)
        self.shapes = ab.astype(np.float16).view(np.uint16)
        self.E, self.N, self.K, self.bits, self.group = E, N, K, bits, group

    def upload(self):
        packed = pack_fields(self.codes.reshape(self.E * self.N, self.K), self.bits)
        self.weight = cq.CubicWeight(torch.from_numpy(packed).to(DEV).reshape(-1),
                                     torch.from_numpy(self.scales).to(DEV).reshape(-1),
                                     torch.from_numpy(self.shapes.view(np.int16)).to(DEV).reshape(-1), self.N, self.K,
                                     self.bits, self.group)
        return self

    def dense(self, e):
        return oracle.dequant(self.codes[e], self.scales[e], self.shapes[e], self.bits, self.group)

    def parts(self, e):
        """Per code the sum of the magnitudes of its level's three parts (2 bits: the level's)."""
        if self.bits == 2:
            return np.abs(self.dense(e))
        M, K = 1 << (self.bits - 1), (1 << (self.bits - 1)) - 1
        n = np.abs(self.codes[e].astype(np.float64))
        rep = lambda v: np.repeat(v, self.group, axis=1)
        s = rep(self.scales[e].astype(np.float64))
        ab = self.shapes[e].view(np.float16).astype(np.float64)
        a, b = rep(ab[..., 0]), rep(ab[..., 1])
        c = 1.0 - a - b
        return s * (np.abs(a / K + M * b / K ** 2 + M * M * c / K ** 3) * n
                    + np.abs(b / K ** 2 + 1.5 * M * c / K ** 3) * n * (M - n)
                    + np.abs(c / K ** 3) * np.abs(n * (M - n) * (n - M / 2)))


def _silu(g):
    return g / (1.0 + np.exp(-g))


def _sum_bound(x, parts):
    """Bound of a row's fp32 sum over x [K] and levels with part magnitudes [N][K]."""
    K = x.size
    block = np.abs(x).reshape(-1, 256 if K % 256 == 0 else 128).max(axis=1)
    fixed = 2.0 ** -30 * np.repeat(block, K // block.size)
    return (3 * K / 128 + 24) * U * (parts @ np.abs(x)) + parts @ fixed


def _reference(x, ids, weights, gu, dn):
    """(y float64 [T][H], its elementwise bound)."""
    X = oracle.bf16_bits_to_f64(x_bits(x))
    T, H = X.shape
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    cache = {}
    for t in range(T):
        for e, w in zip(ids[t], weights[t]):
            if e not in cache:
                cache[e] = gu.dense(e), gu.parts(e), dn.dense(e), dn.parts(e)
            G, Gp, D, Dp = cache[e]
            I = D.shape[1]
            s, d = G @ X[t], _sum_bound(X[t], Gp)
            g, u, dg, du = s[:I], s[I:], d[:I], d[I:]
            v = _silu(g) * u
            h = oracle.bf16_rne(v)
            # |SiLU'| < 1.1
            dv = 1.1 * dg * (np.abs(u) + du) + (np.abs(_silu(g)) + 1.1 * dg) * du + 2.0 ** -20 * np.abs(v)
            dh = np.maximum(np.abs(oracle.bf16_rne(v + dv) - h), np.abs(oracle.bf16_rne(v - dv) - h))
            y[t] += w * (D @ h)
            bound[t] += abs(w) * (np.abs(D) @ dh + _sum_bound(np.abs(h) + dh, Dp)) + 4 * U * abs(w) * (np.abs(D) @ np.abs(h))
    return y, bound + 2.0 ** -140


def _check(x, gu, dn, topk, seed):
    T = x.shape[0]
    logits = torch.randn((T, gu.E), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    y, ids, w = cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, gu.E, topk, out_dtype=torch.float32)
    y = y.cpu().numpy().astype(np.float64)
    ref, bound = _reference(x, ids.cpu().numpy(), w.cpu().numpy().astype(np.float64), gu, dn)
    over = np.abs(y - ref) / bound
    assert np.isfinite(y).all() and over.max() <= 1.0, f"{over.max():.1f} times the bound"
    return np.linalg.norm(y - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("bits,group", [(2, 256), (2, 128), (3, 128), (4, 256)])
@pytest.mark.parametrize("T", [1, 4, 8])
def test_small_activations_beside_outliers(T, bits, group):
    """Outliers 2^13 above the rest where every gate and up code is zero, and h values some 2^12 above
    the rest where every down code is zero: the rest keeps its own precision."""
    say(f"layer beside outliers bits={bits} group={group} T={T}")
    H, I, E = 1024, 512, 4
    gu, dn = Experts(T, E, 2 * I, H, bits, group), Experts(T + 1, E, H, I, bits, group)
    gu.codes[:, :, 5::64] = 0
    large = np.r_[7:I:64, I + 7:2 * I:64]
    gu.scales[:, large] *= 64.0
    dn.codes[:, :, 7::64] = 0
    x = torch.randn((T, H), generator=torch.Generator(device=DEV).manual_seed(bits), device=DEV)
    x[:, 5::64] *= 2.0 ** 13
    _check(x.to(torch.bfloat16), gu.upload(), dn.upload(), 2, 10 * T + bits)


@pytest.mark.parametrize("bits,group", [(2, 256), (2, 128), (3, 128), (4, 256)])
@pytest.mark.parametrize("T", [1, 4, 8])
def test_large_products_that_cancel(T, bits, group):
    """Two equal activations 2^10 above the rest, which every row reads with levels of opposite sign."""
    say(f"layer with cancelling outliers bits={bits} group={group} T={T}")
    H, I, E = 1024, 512, 4
    gu, dn = Experts(T + 30, E, 2 * I, H, bits, group), Experts(T + 31, E, H, I, bits, group)
    k = (1 << (bits - 1)) - 1
    sign = np.random.default_rng(bits).choice([-k, k], size=(E, 2 * I)).astype(np.int8)
    gu.codes[:, :, 40], gu.codes[:, :, 100] = sign, -sign
    x = torch.randn((T, H), generator=torch.Generator(device=DEV).manual_seed(bits), device=DEV)
    x[:, 40] = x[:, 100] = 1.5 * 2.0 ** 10
    _check(x.to(torch.bfloat16), gu.upload(), dn.upload(), 2, 10 * T + bits + 1)


@pytest.mark.parametrize("bits,group", [(2, 512), (2, 128), (3, 256), (4, 128)])
@pytest.mark.parametrize("T", [2, 8])
def test_ordinary_sums(T, bits, group):
    """A hundredth of the channels 20 times larger. Sums' errors add up at random, some 2^-22 of them (rms):
    2^-22 * 2^8 = 2^-14 of the h values round to a neighbour, 2^-8 away (rms, of values alike): 2^-15 =
    3e-5 as a 2-norm, three times as much where a few large h values make up the norm; the bar is 1e-4."""
    say(f"layer, ordinary sums bits={bits} group={group} T={T}")
    H, I, E, topk = 1024, 1024, 12, 8
    gu, dn = Experts(T + 60, E, 2 * I, H, bits, group).upload(), Experts(T + 61, E, H, I, bits, group).upload()
    g = torch.Generator(device=DEV).manual_seed(bits)
    x = torch.randn((T, H), generator=g, device=DEV)
    x[:, torch.rand((H,), generator=g, device=DEV) < 0.01] *= 20.0
    assert _check(x.to(torch.bfloat16), gu, dn, topk, T) <= 1e-4


@pytest.mark.parametrize("bits", [3, 4])
def test_non_finite_rows_of_wide_codes(bits):
    say(f"layer, non-finite activations, bits={bits}")
    gu, dn = Experts(1, 6, 512, 512, bits, 256).upload(), Experts(2, 6, 512, 256, bits, 128).upload()
    for T in (2, 4, 7):
        x = torch.randn((T, 512), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).to(torch.bfloat16)
        logits = torch.randn((T, 6), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV)
        want = cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, 6, 3, out_dtype=torch.float32)[0].cpu().numpy()
        bad = x.clone()
        bad[1, 300] = float("nan") if T != 4 else float("-inf")
        got = cq.cubic_moe_layer(bad, logits, gu.weight, dn.weight, 6, 3, out_dtype=torch.float32)[0].cpu().numpy()
        assert not np.isfinite(got[1]).any()
        keep = [t for t in range(T) if t != 1]
        assert np.array_equal(got[keep], want[keep])
