"""The router's weights are rounded to fp32 once, in every mode: scores, sums and quotients are held in
fp64, whose own errors (some 2^-50) let a weight be off by half a step, 2^-24 of itself, and no more."""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,topk", [(64, 8, 8), (40, 256, 8), (20, 896, 16), (9, 2048, 64)])
def test_weights_round_once(T, E, topk, score, with_bias, renorm):
    say(f"router precision T={T} E={E} topk={topk} {score} bias={with_bias} renorm={renorm}")
    g = torch.Generator(device=DEV).manual_seed(T + E)
    logits = 1.5 * torch.randn((T, E), generator=g, device=DEV)
    logits[1] += 60.0                            # far from zero
    logits[2] *= 30.0                            # one score near one, the others tiny
    logits[3, E // 2:] = -float("inf")
    logits[4] = 0.25                             # all alike
    bias = 0.1 * torch.randn((E,), generator=g, device=DEV) if with_bias else None
    ids, w = cq.cubic_moe_topk(logits, topk, score=score, bias=bias, renormalize=renorm)
    ref_ids, ref = oracle.moe_topk(logits.double().cpu().numpy(), topk, score,
                                   None if bias is None else bias.cpu().numpy(), renorm)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    off = np.abs(w.cpu().numpy().astype(np.float64) - ref)
    assert (off <= 2.0 ** -24 * (1 + 1e-6) * np.abs(ref) + 2.0 ** -149).all(), (off / np.maximum(ref, 1e-300)).max() * 2.0 ** 24
