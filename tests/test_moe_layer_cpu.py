"""The router and the routed-expert layer without a GPU: the oracle's router against an exact
brute force, size queries, and the refusals that the library returns before any launch."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import dequant_gemm_amd as cq
import oracle

OK, ERR_NULL, ERR_SHAPE, ERR_BITS, ERR_GROUP, ERR_ALIGN, ERR_WS, ERR_DTYPE, ERR_OPTION = (
    0, -1, -2, -3, -4, -5, -7, -9, -10)
P16, P8 = ctypes.c_void_p(16), ctypes.c_void_p(8)


def _router(logits=16, bias=None, dtype=0, E=8, topk=2, score=0, renorm=1, scale=1.0):
    return cq._CRouter(logits, bias, dtype, E, topk, score, renorm, scale)


def _w(N=256, K=512, bits=2, group=256, codes=16):
    return cq._CWeight(codes, 16, 16, N, K, bits, group)


def test_oracle_router_order_ties_and_masks():
    inf, nan = np.inf, np.nan
    L = np.array([[1.0, 3.0, 3.0, 2.0, -1.0],
                  [-inf, 0.0, nan, -inf, -5.0],
                  [nan, -inf, nan, -inf, -inf],
                  [inf, 1.0, inf, 0.0, 0.0],
                  [0.0, -0.0, 0.0, -0.0, 0.0]])
    ids, w = oracle.moe_topk(L, 3, "softmax")
    assert ids.tolist() == [[1, 2, 3], [1, 4, -1], [-1, -1, -1], [0, 2, 1], [0, 1, 2]]
    assert np.allclose(w[0], np.exp([3.0, 3.0, 2.0]) / np.exp([3.0, 3.0, 2.0]).sum(), rtol=1e-15)
    assert w[1, 2] == 0 and not w[2].any() and w[3].tolist() == [0.5, 0.5, 0.0]
    # a bias moves the selection, not the weights; a bias of -inf keeps an expert out
    ids, w = oracle.moe_topk(L[:1], 2, "sigmoid", bias=[0.0, -inf, 0.0, 0.5, 5.0], renormalize=False, scale=2.0)
    assert ids.tolist() == [[4, 3]]
    assert np.allclose(w[0], 2.0 / (1.0 + np.exp([1.0, -2.0])), rtol=1e-15)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_oracle_router_against_rationals(score):
    """Scores from a rational exponential (Taylor series with a bounded rest), keys compared exactly."""
    def expq(v):
        n, term, total = 0, Fraction(1), Fraction(1)
        half = Fraction(v) / 64
        while n < 30:
            n += 1
            term = term * half / n
            total += term
        return total ** 64

    rng = np.random.default_rng(5)
    L = rng.normal(size=(4, 9)).astype(np.float32)
    bias = (0.2 * rng.normal(size=9)).astype(np.float32)
    ids, w = oracle.moe_topk(L, 4, score, bias=bias)
    for t in range(4):
        e = [expq(float(v)) for v in L[t]]
        p = [v / sum(e) for v in e] if score == "softmax" else [v / (1 + v) for v in e]
        key = [a + Fraction(float(b)) for a, b in zip(p, bias)]
        order = sorted(range(9), key=lambda i: (-key[i], i))[:4]
        assert ids[t].tolist() == order
        total = sum(p[i] for i in order)
        assert np.allclose(w[t], [float(p[i] / total) for i in order], rtol=1e-12)


def test_topk_refusals():
    lib = cq.load_library()
    call = lambda r, T=4, ids=P16, w=P16: lib.cubic_moe_topk(ctypes.byref(r), T, ids, w, None)
    assert lib.cubic_moe_topk(None, 4, P16, P16, None) == ERR_NULL
    assert call(_router(E=0)) == ERR_SHAPE
    assert call(_router(E=2049)) == ERR_SHAPE
    assert call(_router(topk=0)) == ERR_SHAPE
    assert call(_router(topk=9)) == ERR_SHAPE                  # more than the experts
    assert call(_router(E=128, topk=65)) == ERR_SHAPE
    assert call(_router(), T=-1) == ERR_SHAPE
    assert call(_router(), T=1 << 40) == ERR_SHAPE
    assert call(_router(), T=(1 << 25) + 1) == ERR_SHAPE
    assert call(_router(dtype=3)) == ERR_DTYPE
    assert call(_router(score=2)) == ERR_OPTION
    assert call(_router(logits=0)) == ERR_NULL
    assert call(_router(logits=8)) == ERR_ALIGN
    assert call(_router(bias=8)) == ERR_ALIGN
    assert call(_router(), ids=None) == ERR_NULL
    assert call(_router(), w=P8) == ERR_ALIGN
    assert call(_router(logits=0), T=0) == OK                  # no-op
    assert b"option" in lib.cubic_status_string(ERR_OPTION)


def test_layer_refusals_and_workspace():
    lib = cq.load_library()
    T, topk, E, H, I = 4, 2, 8, 512, 256
    need = lib.cubic_moe_layer_workspace_bytes(T, topk, E, H, I)
    up = lambda n: -(-n // 256) * 256
    P = T * topk
    # the routing, then the larger of the two paths' intermediates
    assert need == 2 * up(4 * P) + max(lib.cubic_moe_mlp_workspace_bytes(T, topk, E, H, I),
                                       up(4 * (2 + 2 * P)) + up(2 * P * I) + up(P * 2 * (I // 32)))
    assert lib.cubic_moe_layer_workspace_bytes(-1, topk, E, H, I) == 0
    assert lib.cubic_moe_layer_workspace_bytes(T, 0, E, H, I) == 0
    gu, dn = _w(N=2 * I, K=H), _w(N=H, K=I)

    def call(r=None, gu=gu, dn=dn, T=T, x=P16, y=P16, yd=1, ws=P16, n=need, ids=None, w=None):
        r = r or _router()
        return lib.cubic_moe_layer(x, T, ctypes.byref(r), ctypes.byref(gu), ctypes.byref(dn), y, yd, ids, w, ws, n,
                                   None)
    assert call(T=0, ws=None, n=0) == OK
    assert call(_router(topk=9)) == ERR_SHAPE
    assert call(_router(score=7)) == ERR_OPTION
    assert call(_router(dtype=-1)) == ERR_DTYPE
    assert call(yd=2) == ERR_DTYPE
    assert call(gu=_w(N=2 * I + 16, K=H)) == ERR_SHAPE
    assert call(dn=_w(N=H + 128, K=I)) == ERR_SHAPE
    assert call(gu=_w(N=2 * I, K=H, bits=1)) == ERR_BITS
    assert call(gu=_w(N=2 * I, K=H, group=64)) == ERR_GROUP
    assert call(gu=_w(N=2 * I, K=H, codes=0)) == ERR_NULL
    assert call(x=None) == ERR_NULL and call(y=None) == ERR_NULL and call(ws=None) == ERR_NULL
    assert call(x=P8) == ERR_ALIGN and call(ids=P8) == ERR_ALIGN and call(w=P8) == ERR_ALIGN
    assert call(n=64) == ERR_WS
    assert call(T=9, n=need) == ERR_WS                          # the composed path needs more
    assert lib.cubic_moe_layer(P16, T, None, ctypes.byref(gu), ctypes.byref(dn), P16, 1, None, None, P16, need,
                               None) == ERR_NULL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        cq.cubic_moe_topk(torch.zeros(2, 8), 2)
    with pytest.raises(TypeError):
        cq.cubic_moe_topk(torch.zeros(2, 8, dtype=torch.float64), 2)
