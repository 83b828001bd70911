"""The gated block's forward pass of up to 64 rows on both sides of every border between the streaming kernel and the
tiles, within the tolerances of the operator's own tests; its workspace follows the same choice."""
import pytest
import torch

import dequant_gemm_amd as cq
from tests import test_gpu_gated_ff as ff
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu


# rows and sizes of the streaming kernel, then those of the tiles, each beside the border
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,H,I", [(4, 72, 8200), (5, 264, 6144), (16, 136, 6144), (32, 72, 4096), (33, 4096, 264), (64, 4096, 72), (64, 136, 4096),
                                   (5, 264, 6152), (16, 136, 6152), (17, 72, 4104), (32, 264, 4104), (33, 4104, 264), (64, 8192, 136), (64, 136, 4104), (48, 4104, 8)])
def test_forward_of_few_rows(M, H, I, dtype):
    act = "silu" if dtype == torch.bfloat16 else "gelu_tanh"
    say(f"gated_ff M={M} H={H} I={I} {act} {dtype}")
    x, w, _ = ff._data(M + H, M, H, I, dtype)
    h, guard = ff._guarded((M, I), dtype)
    pre, guard_p = ff._guarded((M, 2 * I), torch.float32)
    n = cq.cubic_gated_ff_workspace_bytes(M, H, I)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    cq.cubic_gated_ff(x, w, act=act, out=h, pre=pre, workspace=ws[:max(n, 1)])
    assert bool(torch.isnan(guard).all()) and bool(torch.isnan(guard_p).all()) and bool((ws[n:] == 0xFF).all())
    ff._check_h(h, pre, x, w, act, dtype)
    alone = cq.cubic_gated_ff(x, w, act=act)
    assert torch.equal(alone.view(torch.int16), h.view(torch.int16))
