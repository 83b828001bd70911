"""The gate's activation and its slope at every fp16 value: gate and up (one) exact, so that h and the gradients are
the activation and its slope rounded once.

Tolerances: the logistic within 2^-21 + |z| 2^-23 of itself (the hardware's exp2 and reciprocal, an argument rounded
twice), GELU's z another |z| 2^-22 (three roundings); a product's and a sum's rounding; half a step of
fp16, of the value's own binade. Beyond |z| = 88, where exp leaves fp32, values of at most |g| 2^-126."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu


def _gates():
    b = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    return b[torch.isfinite(b)].sort()[0]


@pytest.mark.parametrize("M", [1, 70])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_every_fp16_gate(act, M):
    say(f"activation of every fp16 value {act} M={M}")
    g = _gates()
    g = torch.cat([g, torch.zeros(-g.numel() % 8, dtype=torch.float16)])
    I = g.numel()
    w = torch.zeros((2 * I, 8), dtype=torch.float16)
    w[:I, 0], w[I:, 0] = g, 1.0
    x = torch.zeros((M, 8), dtype=torch.float16)
    x[:, 0] = 1.0
    h, pre = cq.cubic_gated_ff(x.to(DEV), w.to(DEV), act=act, save_pre=True)
    gd = g.double().numpy()
    assert np.array_equal(pre[M - 1, :I].double().cpu().numpy(), gd) and bool((pre[:, I:] == 1).all())
    value, slope = oracle.act_and_slope(gd, act)
    z = gd if act == "silu" else 2 * np.sqrt(2 / np.pi) * (gd + 0.044715 * gd ** 3)
    far = np.minimum(np.abs(z), 100)
    off = 2.0 ** -21 + far * 2.0 ** -23 + (0.0 if act == "silu" else far * 2.0 ** -22)

    def half(v):
        with np.errstate(divide="ignore"):
            return np.exp2(np.maximum(np.floor(np.log2(np.abs(v))), -14.0) - 11) * (1 + 2.0 ** -12)

    tol = (off + 2.0 ** -23) * np.abs(value) + half(value) + np.abs(gd) * 2.0 ** -126
    err = np.abs(h.double().cpu().numpy() - value[None])
    assert (err <= tol[None]).all(), (err / tol[None]).max()
    # slopes: dh = 1, x one-hot: the weight's gradient of a single row is dg itself
    if M == 1:
        dh = torch.ones((1, I), dtype=torch.float16, device=DEV)
        _, dw = cq.cubic_gated_ff_backward(dh, x.to(DEV), w.to(DEV), pre, act=act, need_dx=False)
        p = 1 / (1 + np.exp(np.minimum(-z, 700)))
        bend = np.abs(slope - p)                      # p (1 + g q) = p + g p q, or p + g p q z'
        # dg and du are rounded to eleven bits before the result is, which counts where that has fewer
        twice = lambda v: half(v) + np.where(np.abs(v) < 2.0 ** -14, 2.0 ** -11 * np.abs(v), 0.0)  # noqa: E731
        want = (off + 2.0 ** -20) * (p + bend) + twice(slope) + 2.0 ** -120
        err = np.abs(dw[:I, 0].double().cpu().numpy() - slope)
        assert (err <= want).all(), (err / want).max()
        want = (off + 2.0 ** -23) * np.abs(value) + twice(value) + np.abs(gd) * 2.0 ** -126
        err = np.abs(dw[I:, 0].double().cpu().numpy() - value)
        assert (err <= want).all(), (err / want).max()
