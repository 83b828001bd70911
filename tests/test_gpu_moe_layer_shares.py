"""The routed-expert layer with rows that the first kernel takes in several launches (their activations do
not fit in LDS at once), whose sums go through the workspace: every kind of code, the unused field,
masked and non-finite rows, graphs and streams.

Bars: sums are exact in steps and added up in fp32, so y is off by single h values that round to a
neighbour: with some 2^-22 of a sum, 2^-14 of them (2^-15 as a 2-norm), and where one of few h values
makes up much of a row, 2^-8 of that row; 1e-3 holds both.
"""
import numpy as np
import pytest
import torch

import dequant_gemm_amd as cq
import oracle
from tests._gpu import DEV, pack_fields, say, x_bits

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Experts:
    def __init__(self, seed, E, N, K, bits, group, unused=0.0):
        rng = np.random.default_rng(seed)
        km = (1 << (bits - 1)) - 1
        codes = rng.integers(-km, km + 1, size=(E, N, K)).astype(np.int8)
        if unused:
            codes[rng.random(codes.shape) < unused] = -km - 1
        scales = (0.01 * np.exp(0.3 * rng.normal(size=(E, N, K // group)))).astype(np.float32)
        ab = np.stack([rng.uniform(0.6, 1.4, scales.shape), rng.uniform(-0.1, 0.2, scales.shape)], axis=-1)
        shapes = ab.astype(np.float16).view(np.uint16)
        self.E, self.parts, self.bits, self.group = E, (codes, scales, shapes), bits, group
        self.weight = cq.CubicWeight(torch.from_numpy(pack_fields(codes.reshape(E * N, K), bits)).to(DEV).reshape(-1),
                                     torch.from_numpy(scales).to(DEV).reshape(-1),
                                     torch.from_numpy(shapes.view(np.int16)).to(DEV).reshape(-1), N, K, bits, group)

    def dense(self, e):
        c, s, a = (v[e] for v in self.parts)
        return oracle.dequant(c, s, a, self.bits, self.group)


def _inputs(seed, T, H, E):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16),
            torch.randn((T, E), generator=g, device=DEV))


def _call(x, logits, gu, dn, topk, **kw):
    return cq.cubic_moe_layer(x, logits, gu.weight, dn.weight, gu.E, topk, out_dtype=torch.float32, **kw)


def _check(x, logits, gu, dn, topk):
    T, H = x.shape
    n = cq.cubic_moe_layer_workspace_bytes(T, topk, gu.E, H, dn.weight.K)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    y, ids, w = _call(x, logits, gu, dn, topk, workspace=ws[:n])
    assert bool((ws[n:] == 0xFF).all())
    ref, rids, rw = oracle.moe_layer(x_bits(x), logits.double().cpu().numpy(), topk, "softmax", gu.dense, dn.dense)
    assert np.array_equal(ids.cpu().numpy(), rids) and np.allclose(w.cpu().numpy(), rw, rtol=2.0 ** -23, atol=0)
    y = y.cpu().numpy()
    assert np.linalg.norm(y - ref) <= 1e-3 * np.linalg.norm(ref)
    assert np.array_equal(y, _call(x, logits, gu, dn, topk)[0].cpu().numpy())
    return y


@pytest.mark.parametrize("H,T,bits,group", [(5120, 8, 2, 512), (8192, 7, 2, 256), (9216, 5, 2, 384), (12288, 4, 2, 1024),
                                            (20480, 3, 2, 128), (6144, 8, 3, 128), (9216, 6, 4, 256), (16384, 3, 4, 512),
                                            (40960, 1, 3, 256), (65536, 2, 2, 512)])
def test_long_rows(H, T, bits, group):
    say(f"layer shares H={H} T={T} bits={bits} group={group}")
    E, topk, I = 3, 2, 128
    for unused in (0.0, 0.02, 1e-5):             # (1e-5: in single places)
        gu, dn = Experts(H + T, E, 2 * I, H, bits, group, unused), Experts(T, E, H, I, bits, 128, unused)
        x, logits = _inputs(T, T, H, E)
        _check(x, logits, gu, dn, topk)
        if bits != 2 and not unused:
            break


def test_masked_and_non_finite_rows():
    say("layer shares, masked and non-finite rows")
    H, I, E, T = 8192, 128, 4, 8
    gu, dn = Experts(1, E, 2 * I, H, 2, 512), Experts(2, E, H, I, 2, 128)
    x, logits = _inputs(3, T, H, E)
    want = _check(x, logits, gu, dn, 2)
    logits2, bad = logits.clone(), x.clone()
    bad[2, 17], bad[5, 8000] = NAN, float("inf")   # in the first launch's share, and in the last one's
    y = _call(bad, logits, gu, dn, 2)[0].cpu().numpy()
    assert not np.isfinite(y[[2, 5]]).any()
    keep = [0, 1, 3, 4, 6, 7]
    assert np.array_equal(y[keep], want[keep])
    logits2[:] = -float("inf")
    y, ids, w = _call(bad, logits2, gu, dn, 2)
    assert not y.any() and bool((ids == -1).all()) and not w.any()


def test_graph_and_streams():
    """A captured layer replayed on new inputs between eager calls, and two streams with workspaces of their
    own; the captured workspace is overwritten between the replays."""
    say("layer shares in a graph and on two streams")
    H, I, E, T, topk = 8192, 128, 6, 8, 3
    gu, dn = Experts(4, E, 2 * I, H, 2, 512), Experts(5, E, H, I, 2, 128)
    ins = [_inputs(s, T, H, E) for s in range(4)]
    want = [_call(x, l, gu, dn, topk)[0].cpu().numpy() for x, l in ins]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i, (x, l) in enumerate(ins):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(_call(x, l, gu, dn, topk)[0])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy(), w)
    x, l = ins[0][0].clone(), ins[0][1].clone()
    out = torch.empty((T, H), device=DEV)
    ws = torch.empty(cq.cubic_moe_layer_workspace_bytes(T, topk, E, H, I), dtype=torch.uint8, device=DEV)
    _call(x, l, gu, dn, topk, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(x, l, gu, dn, topk, out=out, workspace=ws)
    for i in (1, 2, 3, 0, 2):
        x.copy_(ins[i][0])
        l.copy_(ins[i][1])
        out.fill_(NAN)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want[i])
        assert np.array_equal(_call(*ins[i], gu, dn, topk)[0].cpu().numpy(), want[i])
