"""The routed-expert layer where it runs as the router followed by the MLP step: wide codes, more than 64
tokens, more than 1024 experts. There the products of codes of three bits and more take levels of two bf16
halves, off by 2^-18.5 (rms), where fp16 levels would be off by 2^-13.

A 2-norm bar of 4e-4 tells them apart: an error d of g and u moves v = SiLU(g) u by about 1.4 d, and
v lies 2^7.5 steps of bf16 from zero, so 0.8 * 1.4 d * 2^7.5 of the h values round to a neighbour,
2^-7.5 away. Two halves: 5e-4 of them and sqrt(5e-4) * 2^-7.5 = 1.3e-4 of y (three times that where few h
values make up the norm); fp16: 2.5e-2 of them and 9e-4.
"""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, say, x_bits

pytestmark = pytest.mark.gpu


class Experts:
    def __init__(self, seed, E, N, K, bits, group):
        g = torch.Generator(device=DEV).manual_seed(seed)
        km = (1 << (bits - 1)) - 1
        self.codes = torch.randint(-km, km + 1, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
        self.scales = 0.02 * torch.exp(0.3 * torch.randn((E, N, K // group), generator=g, device=DEV))
        ab = torch.rand((E, N, K // group, 2), generator=g, device=DEV)
        ab = ab * torch.tensor([0.8, 0.3], device=DEV) + torch.tensor([0.6, -0.1], device=DEV)
        self.shapes = ab.to(torch.float16).view(torch.int16)
        self.bits, self.group = bits, group
        self.weight = cq.CubicWeight(cq.cubic_pack(self.codes.reshape(E * N, K), bits).reshape(-1),
                                     self.scales.reshape(-1), self.shapes.reshape(-1), N, K, bits, group)

    def dense(self, e):
        return oracle.dequant(self.codes[e].cpu().numpy(), self.scales[e].cpu().numpy(),
                              self.shapes[e].cpu().numpy().view(np.uint16), self.bits, self.group)


def _check(T, H, I, E, topk, up, down, seed):
    gu, dn = Experts(seed, E, 2 * I, H, *up), Experts(seed + 1, E, H, I, *down)
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=DEV)
    x[:, torch.rand((H,), generator=g, device=DEV) < 0.01] *= 20.0
    x = x.to(torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device=DEV)
    y, ids, w = cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, E, topk, score="sigmoid", out_dtype=torch.float32)
    ref, rids, rw = oracle.moe_layer(x_bits(x), logits.double().cpu().numpy(), topk, "sigmoid", gu.dense, dn.dense)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.allclose(w.cpu().numpy(), rw, rtol=2.0 ** -23, atol=0)
    err = np.linalg.norm(y.cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err <= 4e-4, err


@pytest.mark.parametrize("up,down", [((5, 256), (5, 128)), ((6, 128), (6, 256)), ((7, 256), (7, 128)),
                                     ((8, 128), (8, 256)), ((3, 128), (5, 256)), ((7, 512), (4, 128)),
                                     ((2, 256), (7, 128)), ((8, 128), (2, 256)), ((5, 128), (3, 128))])
@pytest.mark.parametrize("T", [1, 16])
def test_wide_codes(T, up, down):
    say(f"layer composed bits {up}/{down} T={T}")
    _check(T, 512, 512, 8, 4, up, down, 100 * T + 10 * up[0] + down[0])


@pytest.mark.parametrize("bits,group", [(3, 128), (3, 256), (4, 128), (4, 512)])
def test_many_tokens(bits, group):
    say(f"layer composed bits={bits} group={group} T=65")
    _check(65, 512, 512, 6, 2, (bits, group), (bits, 128), bits)


@pytest.mark.parametrize("bits", [3, 4])
def test_many_experts(bits):
    say(f"layer composed bits={bits} E=1025")
    _check(12, 256, 256, 1025, 8, (bits, 128), (bits, 256), bits + 50)
