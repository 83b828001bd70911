"""The quantiser's codes byte for byte, signs of zeros among them: a code has its value's sign, also where it rounds
to zero; blocks of zeros have scale 0 and codes of +0 (the rule of the oracle, which takes the quotient's sign bit)."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu


def _signed_zeros(M, K, dtype, size, seed):
    """Rows around `size` with zeros of both signs and values that round to zero codes in every block, the
    first 128 channels of the first 128 rows zeros of both signs alone."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((M, K), generator=g, device=DEV) * size
    pick = torch.randint(0, 8, (M, K), generator=g, device=DEV)
    x = torch.where(pick == 0, 0.0, torch.where(pick == 1, -0.0, torch.where(pick == 2, x * 2.0 ** -12, x)))
    x[:128, :128] = torch.where(pick[:128, :128] < 4, 0.0, -0.0)
    return x.to(dtype)


# scales of 2^-9 to 2^-7 and of both ends of the bf16 range, which take the division
@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, 1.0), (torch.float16, 1.0), (torch.float16, 2.0 ** -16), (torch.bfloat16, 2.0 ** -100),
                                        (torch.bfloat16, 2.0 ** 115)])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 48), (5, 400), (200, 272), (260, 1040)])
def test_codes_byte_for_byte(M, K, rows, dtype, size):
    say(f"quant_fp8 signed zeros M={M} K={K} rows={rows} {dtype} {size}")
    x = _signed_zeros(M, K, dtype, size, M + K)
    q, s = cq.cubic_quant_fp8(x, rows)
    qr, sr = oracle.quant_fp8(x.double().cpu().numpy(), rows)
    assert np.array_equal(s.cpu().numpy(), sr) and (M < 128 or sr[0, 0] == 0)
    got = q.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, qr), np.argwhere(got != qr)[:4]
    assert (qr == 0x80).any() or K == 48          # the case has what it is about


@pytest.mark.parametrize("dtype,steps", [(torch.bfloat16, 128), (torch.float16, 1024)])
def test_every_pair_of_significands(dtype, steps):
    """Quotients of every significand of a block's largest magnitude and every significand of a value, down to
    codes of zero, against IEEE division on the CPU: scales and codes equal."""
    say(f"quant_fp8 every pair of significands {dtype}")
    sig = 1 + torch.arange(steps, dtype=torch.float32) / steps
    per = -(-steps // 127)                            # blocks of 127 values and the largest magnitude
    for k in range(20):
        v = torch.zeros(per * 127)
        v[:steps] = sig * 2.0 ** -k
        x = torch.empty((steps, per, 128))
        x[:, :, 0] = 1024 * sig[:, None]
        x[:, :, 1:] = 1024 * v.view(per, 127) * torch.where(torch.arange(127) % 2 == 0, 1.0, -1.0)
        if k == 0:                                    # no value above its block's largest magnitude
            x[:, :, 1:] = torch.where(x[:, :, 1:].abs() > x[:, :, :1], 0.0, x[:, :, 1:])
        x = x.view(steps, -1).to(dtype)
        q, s = cq.cubic_quant_fp8(x.to(DEV))
        want_s = (x[:, ::128].float() / 448.0)
        quotient = (x.float().view(steps, per, 128) / want_s[:, :, None]).clamp(-448, 448)
        want = quotient.to(torch.float8_e4m3fn).view(torch.uint8).view(steps, -1)
        assert torch.equal(s.cpu(), want_s), k
        assert torch.equal(q.cpu().view(torch.uint8), want), k
