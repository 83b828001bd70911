"""The backward pass's workspace: large gradients are held once, small ones twice (fp16 scales them for each product)."""
import pytest

import dequant_gemm_amd as cq

align = lambda n: -(-n // 256) * 256  # noqa: E731


@pytest.mark.parametrize("M,H,I,copies", [(4096, 7168, 2048, 1), (16384, 4096, 8192, 1), (4, 64, 64, 2), (256, 512, 256, 2)])
def test_size(M, H, I, copies):
    held = copies * align(M * I * 4) + align((M + 2 * I) * 4)
    need = cq.cubic_gated_ff_backward_workspace_bytes(M, H, I)
    slices = need - held                              # fp32 sums of sliced products: of dx, of dw, two of each at least
    assert slices == 0 or (M * I < 1 << 20 and slices >= min(2 * M * H * 4, 2 * 2 * I * H * 4))
