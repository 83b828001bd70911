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
