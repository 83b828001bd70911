"""Measured cases of three operators of a routed-expert layer served for decoding.

* ``topk``   the router: scores of a token's logits, its top experts and their weights.
* ``layer``  the whole routed-expert layer for a few tokens: router, gate_up product, SiLU(gate) * up,
             down product and the router-weighted sum, on CubicQuant-coded expert weights.
* ``w8a8``   products of per-token int8 activations with per-channel int8 weights (the dense
             projections and shared experts that stay beside the routed experts), from quantised
             activations (``form`` = "gemm") or from bf16 ones quantised on the way ("linear").

Every operator has a plain form in elementary torch operations; with ``own`` set, ``run`` makes the
calls of ``dequant_gemm_amd`` instead.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
FLOAT_MAX = torch.finfo(torch.float32).max
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decoding token's router over the 896 experts of a large layer (sigmoid scores, a selection bias)
        dict(name="topk_1_e896", op="topk", T=1, E=896, topk=16, score="sigmoid", bias=True, renorm=True,
             scale=2.5, dtype="f32", masked=0.0),
        # a decoding batch with softmax scores on bf16 logits (exact ties occur)
        dict(name="topk_64_e256_bf16", op="topk", T=64, E=256, topk=8, score="softmax", bias=False, renorm=True,
             scale=1.0, dtype="bf16", masked=0.0),
        # a prefill chunk's router
        dict(name="topk_4096_e896", op="topk", T=4096, E=896, topk=16, score="sigmoid", bias=True, renorm=True,
             scale=2.5, dtype="f32", masked=0.0),
        # odd sizes, experts masked out (some rows keep fewer experts than slots, or none)
        dict(name="topk_333_e61_masked", op="topk", T=333, E=61, topk=5, score="softmax", bias=True, renorm=False,
             scale=1.0, dtype="f32", masked=0.9),
        # the smallest layer (hidden 512, intermediate 256, 8 experts, top-2), where launches count
        dict(name="layer_mini_t4", op="layer", T=4, H=512, I=256, E=8, topk=2, bits=2, group=256, score="softmax",
             bias=False, out="bf16"),
        # one decoding token through 16 experts of the large layer
        dict(name="layer_k7168_t1", op="layer", T=1, H=7168, I=3072, E=64, topk=16, bits=2, group=512,
             score="sigmoid", bias=True, out="bf16"),
        # a few decoding tokens through the large layer
        dict(name="layer_k7168_t4", op="layer", T=4, H=7168, I=3072, E=128, topk=16, bits=2, group=512,
             score="sigmoid", bias=True, out="bf16"),
        # 4-bit expert weights with groups of 128
        dict(name="layer_w4_t2", op="layer", T=2, H=2048, I=1024, E=32, topk=4, bits=4, group=128, score="sigmoid",
             bias=True, out="bf16"),
        # one decoding token through a dense projection
        dict(name="w8a8_linear_m1", op="w8a8", form="linear", M=1, N=6144, K=7168, out="bf16", bias=False),
        # odd and ragged sizes, a bias, fp32 results
        dict(name="w8a8_linear_m37_odd", op="w8a8", form="linear", M=37, N=1003, K=1928, out="f32", bias=True),
        # a decoding batch
        dict(name="w8a8_gemm_m64", op="w8a8", form="gemm", M=64, N=7168, K=2048, out="bf16", bias=False),
        # a prefill chunk
        dict(name="w8a8_gemm_m4096", op="w8a8", form="gemm", M=4096, N=6144, K=7168, out="bf16", bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "layer", "w8a8"])
    if op == "topk":
        E = _log_int(rng, 8, 1024)
        return dict(op=op, T=_log_int(rng, 1, 3500), E=E, topk=rng.randint(1, min(16, E)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "f32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.9]))
    if op == "layer":
        bits = rng.choice([2, 2, 2, 3, 4])
        group = rng.choice([256, 512]) if bits == 2 else rng.choice([128, 256])
        while True:
            H = group * max(1, _log_int(rng, 512, 7168) // group)
            I = group * max(1, _log_int(rng, 256, 2560) // group)
            E = _log_int(rng, 8, 128)
            T, topk = _log_int(rng, 1, 16), rng.randint(1, min(16, E))
            # expert weights of at most 1.5 G codes, and no more pairs' products than the largest listed case
            if 3 * H * I * E <= 1_500_000_000 and T * topk * H * I <= 16 * 7168 * 3072:
                break
        return dict(op=op, T=T, H=H, I=I, E=E, topk=topk, bits=bits, group=group,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, out="bf16")
    while True:
        M, N, K = _log_int(rng, 1, 4096), _log_int(rng, 16, 8192), 8 * _log_int(rng, 8, 1024)
        if M * N * K <= 4096 * 6144 * 7168:
            break
    return dict(op=op, form=rng.choice(["gemm", "linear"]), M=M, N=N, K=K, out=rng.choice(["bf16", "f32"]),
                bias=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _logits(g, T, E, dtype, masked):
    logits = 1.5 * torch.randn((T, E), generator=g, device=DEVICE)
    if masked:
        # the share of masked experts grows along the rows: none in the first, all in the last
        share = torch.linspace(0.0, 1.0, T, device=DEVICE)[:, None] ** (1.0 - masked) if T > 1 else masked
        logits = logits.masked_fill(torch.rand((T, E), generator=g, device=DEVICE) < share, -math.inf)
    return logits.to(DTYPES[dtype])


def _activations(g, M, K):
    """bf16 rows with a hundredth of the channels twenty times larger, as language models have them."""
    x = torch.randn((M, K), generator=g, device=DEVICE)
    outlier = torch.rand((K,), generator=g, device=DEVICE) < 0.01
    return torch.where(outlier, 20.0 * x, x).to(torch.bfloat16)


def _pack(codes, bits):
    """int codes [..., K] to the LSB-first bit stream, uint8 [..., K * bits / 8]."""
    fields = codes.to(torch.uint8) if bits == 8 else (codes & ((1 << bits) - 1)).to(torch.uint8)
    planes = torch.stack([(fields >> b) & 1 for b in range(bits)], dim=-1)
    planes = planes.reshape(*codes.shape[:-1], -1, 8)
    weights = torch.tensor([1 << b for b in range(8)], dtype=torch.uint8, device=codes.device)
    return (planes * weights).sum(dim=-1, dtype=torch.uint8)


def _experts(g, E, N, K, bits, group):
    """(codes, scales, shapes) of E back-to-back expert matrices [N][K]."""
    if bits == 2:  # P(0) = 1/2, P(+1) = P(-1) = 1/4: random bytes, the unused field 10 read as 00
        raw = torch.randint(0, 256, (E * N * K // 4,), generator=g, device=DEVICE, dtype=torch.uint8)
        codes = raw & ~(raw & ~(raw << 1) & 0xAA)
    else:
        kmax = (1 << (bits - 1)) - 1
        u = torch.rand((E * N, K), generator=g, device=DEVICE) - 0.5
        lap = -0.25 * torch.sign(u) * torch.log1p(-2.0 * u.abs())
        codes = _pack(torch.round(kmax * lap.clamp(-1.0, 1.0)).to(torch.int8), bits).reshape(-1)
    n = E * N * (K // group)
    scales = torch.exp(math.log(0.015) + 0.3 * torch.randn((n,), generator=g, device=DEVICE))
    # increasing curves: the derivative a + 2 b t + 3 c t^2 stays positive over this box
    a = 0.6 + 0.8 * torch.rand((n,), generator=g, device=DEVICE)
    b = 0.3 * torch.rand((n,), generator=g, device=DEVICE) - 0.1
    shapes = torch.stack([a, b], dim=-1).to(torch.float16).view(torch.int16)
    return codes, scales, shapes.reshape(-1)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "topk":
        s["logits"] = _logits(g, case["T"], case["E"], case["dtype"], case["masked"])
        s["router_bias"] = 0.1 * torch.randn((case["E"],), generator=g, device=DEVICE) if case["bias"] else None
    elif case["op"] == "layer":
        T, H, I, E = case["T"], case["H"], case["I"], case["E"]
        s.update(renorm=True, scale=2.5 if case["score"] == "sigmoid" else 1.0)
        s["x"] = _activations(g, T, H)
        s["logits"] = _logits(g, T, E, "f32", 0.0)
        s["router_bias"] = 0.1 * torch.randn((E,), generator=g, device=DEVICE) if case["bias"] else None
        s["gate_up"] = _experts(g, E, 2 * I, H, case["bits"], case["group"])
        s["down"] = _experts(g, E, H, I, case["bits"], case["group"])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        if case["form"] == "linear":
            s["x"] = _activations(g, M, K)
        else:
            s["xq"] = torch.randint(-127, 128, (M, K), generator=g, device=DEVICE, dtype=torch.int8)
            s["x_scale"] = torch.exp(-4.0 + 0.3 * torch.randn((M,), generator=g, device=DEVICE))
        w = torch.randn((N, K), generator=g, device=DEVICE)
        s["w_scale"] = w.abs().amax(dim=1) / 127.0
        s["wq"] = torch.round(w / s["w_scale"][:, None]).clamp(-127, 127).to(torch.int8)
        s["add"] = torch.randn((N,), generator=g, device=DEVICE) if case["bias"] else None
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _plain_topk(logits, bias, topk, score, renorm, scale):
    """ids int32 and weights fp32 [T][topk]: selection by score + bias, ties to the lowest index; experts
    whose logit is NaN or minus infinity are never taken (slots left over: id -1, weight 0)."""
    l = logits.double().clamp(max=FLOAT_MAX)
    gone = torch.isnan(l) | (l == -math.inf)
    l = torch.where(gone, -math.inf, l)
    if score == "softmax":
        top = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        total = e.sum(dim=1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = l if bias is None else p + bias.double()
    order = torch.sort(torch.where(gone, -math.inf, key), dim=1, descending=True, stable=True)[1][:, :topk]
    left = torch.gather(gone, 1, order)
    w = torch.where(left, 0.0, torch.gather(p, 1, order))
    if renorm:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return torch.where(left, -1, order).to(torch.int32), (w * scale).float()


def _plain_weights(experts, ids, N, K, bits, group):
    """fp32 matrices [P][N][K] of the chosen experts."""
    codes, scales, shapes = experts
    packed = codes.view(-1, N, K * bits // 8)[ids]
    bit = torch.arange(K, device=packed.device) * bits
    lo, off = bit // 8, (bit % 8).to(torch.int16)
    hi = torch.clamp(lo + 1, max=K * bits // 8 - 1)
    field = (packed[..., lo].to(torch.int16) | (packed[..., hi].to(torch.int16) << 8)) >> off
    field = field & ((1 << bits) - 1)
    k = torch.where(field >= 1 << (bits - 1), field - (1 << bits), field).float()
    k = k.view(k.shape[0], N, K // group, group)
    s = scales.view(-1, N, K // group, 1)[ids]
    ab = shapes.view(torch.float16).view(-1, N, K // group, 2)[ids].float()
    a, b = ab[..., :1], ab[..., 1:]
    t = k.abs() / float((1 << (bits - 1)) - 1)
    q = t * (a + t * (b + t * (1.0 - a - b)))
    return (s * torch.sign(k) * q).view(k.shape[0], N, K)


def _plain_layer(s):
    T, H, I, topk = s["T"], s["H"], s["I"], s["topk"]
    ids, weights = _plain_topk(s["logits"], s["router_bias"], topk, s["score"], s["renorm"], s["scale"])
    flat = ids.reshape(-1).clamp(min=0).long()
    rows = s["x"].float().repeat_interleave(topk, dim=0)
    gu = _plain_weights(s["gate_up"], flat, 2 * I, H, s["bits"], s["group"])
    gu = torch.matmul(gu, rows[:, :, None])[:, :, 0]
    gate, up = gu[:, :I], gu[:, I:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float()  # the layer keeps h in bf16
    o = torch.matmul(_plain_weights(s["down"], flat, H, I, s["bits"], s["group"]), h[:, :, None])[:, :, 0]
    taken = (ids >= 0)[:, :, None]
    y = torch.where(taken, weights[:, :, None] * o.view(T, topk, H), 0.0).sum(dim=1)
    return {"y": y.to(DTYPES[s["out"]]), "ids": ids, "weights": weights}


def _plain_quantise(x):
    x = x.float()
    scale = x.abs().amax(dim=1) / 127.0
    q = torch.round(x / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-127, 127)
    return q, scale


def _plain_w8a8(s):
    if s["form"] == "linear":
        xq, xs = _plain_quantise(s["x"])
    else:
        xq, xs = s["xq"].float(), s["x_scale"]
    y = torch.matmul(xq, s["wq"].float().t()) * s["w_scale"] * xs[:, None]
    if s["add"] is not None:
        y = y + s["add"]
    return {"y": y.to(DTYPES[s["out"]])}


def _plain(s):
    if s["op"] == "topk":
        ids, weights = _plain_topk(s["logits"], s["router_bias"], s["topk"], s["score"], s["renorm"], s["scale"])
        return {"ids": ids, "weights": weights}
    return _plain_layer(s) if s["op"] == "layer" else _plain_w8a8(s)


# ----------------------------------------------------------------------------------- the framework's calls


def _own(s):
    import dequant_gemm_amd as cq

    if s["op"] == "topk":
        ids, weights = cq.cubic_moe_topk(s["logits"], s["topk"], score=s["score"], bias=s["router_bias"],
                                         renormalize=s["renorm"], scale=s["scale"])
        return {"ids": ids, "weights": weights}
    if s["op"] == "layer":
        T, H, I, E = s["T"], s["H"], s["I"], s["E"]
        if "workspace" not in s:  # kept by a serving program, like the weights' descriptors
            n = cq.cubic_moe_layer_workspace_bytes(T, s["topk"], E, H, I)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEVICE)
            s["experts"] = [cq.CubicWeight(*s[w], N, K, s["bits"], s["group"])
                            for w, N, K in (("gate_up", 2 * I, H), ("down", H, I))]
        y, ids, weights = cq.cubic_moe_layer(s["x"], s["logits"], *s["experts"], E, s["topk"], score=s["score"],
                                             bias=s["router_bias"], renormalize=s["renorm"], scale=s["scale"],
                                             workspace=s["workspace"], out_dtype=DTYPES[s["out"]])
        return {"y": y, "ids": ids, "weights": weights}
    weight = cq.Int8Weight(s["wq"], s["w_scale"])
    if s["form"] == "linear":
        return {"y": cq.cubic_linear_w8a8(s["x"], weight, bias=s["add"], out_dtype=DTYPES[s["out"]])}
    return {"y": cq.cubic_gemm_w8a8(s["xq"], s["x_scale"], weight, bias=s["add"], out_dtype=DTYPES[s["out"]])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work of one pass


def work(case):
    if case["op"] == "topk":
        T, E, k = case["T"], case["E"], case["topk"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4.0 * T * E}
    if case["op"] == "layer":
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["topk"]
        touched = E * (1.0 - (1.0 - k / E) ** T)  # the expected number of experts that any token takes
        stored = 3 * H * I * case["bits"] / 8 + 3 * H * I / case["group"] * 8
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": touched * stored + T * H * (2 + size) + 4 * T * E + 8 * T * k,
                "flops": 2.0 * T * k * 3 * H * I}
    M, N, K = case["M"], case["N"], case["K"]
    read = M * K * (2 if case["form"] == "linear" else 1) + N * K + 4 * N * (2 if case["bias"] else 1)
    return {"bytes": read + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------- the definitions in 64 bits, for reference


def _exact_topk(logits, bias, topk, score, renorm, scale):
    """Row by row in numpy: explicit (key, index) order."""
    l = logits.double().cpu().numpy()
    c = None if bias is None else bias.double().cpu().numpy()
    T, E = l.shape
    ids, weights = np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    for t in range(T):
        live = np.flatnonzero(~np.isnan(l[t]) & (l[t] != -np.inf))
        if not live.size:
            continue
        v = np.minimum(l[t, live], FLOAT_MAX)
        if score == "softmax":
            p = np.exp(v - v.max())
            p /= math.fsum(p)
        else:
            p = np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))
        order = np.lexsort((live, -(v if c is None else p + c[live])))[:topk]
        ids[t, :order.size] = live[order]
        weights[t, :order.size] = p[order]
        if renorm and weights[t].sum() > 0:
            weights[t] /= math.fsum(weights[t])
    return ids, weights * scale


def _exact_matrix(experts, e, N, K, bits, group):
    """Expert e's weights in float64 [N][K], each code put together from its bits."""
    codes, scales, shapes = experts
    size = N * K * bits // 8
    raw = codes[e * size:(e + 1) * size]
    stream = torch.stack([(raw >> b) & 1 for b in range(8)], dim=-1).reshape(N * K, bits)
    code = sum(stream[:, b].to(torch.int16) << b for b in range(bits - 1))
    code = (code - (stream[:, bits - 1].to(torch.int16) << (bits - 1))).reshape(N, K).double()
    n = N * (K // group)
    s = scales[e * n:(e + 1) * n].double().reshape(N, -1).repeat_interleave(group, dim=1)
    ab = shapes[2 * e * n:2 * (e + 1) * n].view(torch.float16).double().reshape(N, -1, 2)
    a, b = (ab[..., i].repeat_interleave(group, dim=1) for i in (0, 1))
    t = code / float((1 << (bits - 1)) - 1)  # odd powers carry the sign, the square takes it explicitly
    return s * (a * t + b * t * t.abs() + (1.0 - a - b) * t ** 3)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w8a8":
        if case["M"] * case["N"] * case["K"] > 1 << 38:
            return None
        if case["form"] == "linear":
            x = s["x"].float()
            xs = x.abs().amax(dim=1) / 127.0  # the scale and the quotient are fp32 by definition
            xq = torch.where(xs[:, None] > 0, x / xs[:, None], 0.0).round().clamp(-127, 127).double()
        else:
            xq, xs = s["xq"].double(), s["x_scale"]
        y = torch.einsum("mk,nk->mn", xq, s["wq"].double())
        y = y * torch.outer(xs.double(), s["w_scale"].double())
        return {"y": y if s["add"] is None else y + s["add"].double()[None, :]}
    if case["op"] == "topk":
        ids, weights = _exact_topk(s["logits"], s["router_bias"], s["topk"], s["score"], s["renorm"], s["scale"])
        return {"ids": ids, "weights": weights}
    T, H, I, topk = s["T"], s["H"], s["I"], s["topk"]
    ids, weights = _exact_topk(s["logits"], s["router_bias"], topk, s["score"], s["renorm"], s["scale"])
    y = torch.zeros((T, H), dtype=torch.float64, device=DEVICE)
    for e in sorted(set(ids.reshape(-1).tolist()) - {-1}):
        gu = _exact_matrix(s["gate_up"], e, 2 * I, H, s["bits"], s["group"])
        down = _exact_matrix(s["down"], e, H, I, s["bits"], s["group"])
        for t, j in zip(*np.nonzero(ids == e)):
            g = gu @ s["x"][t].double()
            h = g[:I] * torch.sigmoid(g[:I]) * g[I:]
            y[t] += weights[t, j] * (down @ h.to(torch.bfloat16).double())
    return {"y": y, "ids": ids, "weights": weights}
