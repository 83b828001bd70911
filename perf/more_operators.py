"""Measured cases of two operators of the dense parts that stay beside routed experts.

* ``fp8``   products of e4m3 activations with one scale per token and 128 channels and e4m3 weights
            with one scale per block of 128 x 128, from quantised activations (``form`` = "gemm") or from
            bf16 ones quantised on the way ("linear").
* ``ff``    the gated feed-forward block h = act(x Wg^T) * (x Wu^T) of a shared expert or a dense layer:
            with bf16 or fp16 weights (``form`` = "plain"), with e4m3 block-scaled ones and activations
            quantised on the way ("fp8"), and as a training step, forward and backward ("step").

Every operator has a plain form in elementary torch operations; with ``own`` set, ``run`` makes the
calls of ``dequant_gemm_amd`` instead.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 128
E4M3_MAX = 448.0
GELU_C, GELU_K = math.sqrt(2.0 / math.pi), 0.044715
LARGEST = 4096 * 6144 * 7168      # products of the largest listed case


def listed():
    return [
        # one decoding token through a dense projection
        dict(name="fp8_linear_m1", op="fp8", form="linear", M=1, N=6144, K=7168, out="bf16", bias=False),
        # odd and ragged sizes (blocks cut at the edges), a bias, fp32 results
        dict(name="fp8_linear_m37_odd", op="fp8", form="linear", M=37, N=1003, K=1936, out="f32", bias=True),
        # a decoding batch
        dict(name="fp8_gemm_m64", op="fp8", form="gemm", M=64, N=7168, K=2048, out="bf16", bias=False),
        # a prefill chunk
        dict(name="fp8_gemm_m4096", op="fp8", form="gemm", M=4096, N=6144, K=7168, out="bf16", bias=False),
        # one decoding token through a shared expert
        dict(name="ff_m1", op="ff", form="plain", M=1, H=7168, I=2048, dtype="bf16", act="silu"),
        # odd sizes, fp16, the other activation
        dict(name="ff_m45_odd", op="ff", form="plain", M=45, H=1000, I=520, dtype="f16", act="gelu_tanh"),
        # a prefill chunk through a shared expert
        dict(name="ff_m4096", op="ff", form="plain", M=4096, H=7168, I=2048, dtype="bf16", act="silu"),
        # a decoding batch through a shared expert with 8-bit weights
        dict(name="ff_fp8_m16", op="ff", form="fp8", M=16, H=7168, I=2048, dtype="bf16", act="silu"),
        # a prefill chunk through the same
        dict(name="ff_fp8_m2048", op="ff", form="fp8", M=2048, H=7168, I=2048, dtype="bf16", act="silu"),
        # training steps: the smallest layer (hidden 512, intermediate 256), odd sizes, a large layer
        dict(name="ff_step_mini", op="ff", form="step", M=256, H=512, I=256, dtype="bf16", act="silu"),
        dict(name="ff_step_m777_odd", op="ff", form="step", M=777, H=1544, I=680, dtype="f16", act="gelu_tanh"),
        dict(name="ff_step_m4096", op="ff", form="step", M=4096, H=7168, I=2048, dtype="bf16", act="silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fp8", "fp8", "plain", "fp8 ff", "step", "step"])
    while True:
        M, wide, K = _log_int(rng, 1, 4096), _log_int(rng, 16, 8192), _log_int(rng, 64, 8192)
        if kind == "fp8":
            case = dict(op="fp8", form=rng.choice(["gemm", "linear"]), M=M, N=wide, K=16 * max(1, K // 16),
                        out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5)
            cost = M * wide * K
        elif kind == "fp8 ff":
            case = dict(op="ff", form="fp8", M=M, H=16 * max(1, K // 16), I=128 * max(1, wide // 256),
                        dtype=rng.choice(["bf16", "bf16", "f16"]), act=rng.choice(["silu", "gelu_tanh"]))
            cost = M * 2 * case["I"] * K
        else:
            case = dict(op="ff", form=kind, M=M, H=8 * max(1, K // 8), I=8 * max(1, wide // 16),
                        dtype=rng.choice(["bf16", "bf16", "f16"]), act=rng.choice(["silu", "gelu_tanh"]))
            cost = M * 2 * case["I"] * K
        if cost <= (LARGEST if kind == "fp8" else 4096 * 4096 * 7168):
            return case


# ---------------------------------------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _activations(g, M, K):
    """fp32 rows with a hundredth of the channels twenty times larger, as language models have them."""
    x = torch.randn((M, K), generator=g, device=DEVICE)
    return torch.where(torch.rand((K,), generator=g, device=DEVICE) < 0.01, 20.0 * x, x)


def _block_weight(g, N, K):
    """A weight of usual size in e4m3 with one scale per block of 128 x 128 (cut at the edges)."""
    w = torch.randn((N, K), generator=g, device=DEVICE) / math.sqrt(K)
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    padded = torch.zeros((nb * BLOCK, kb * BLOCK), device=DEVICE)
    padded[:N, :K] = w
    scales = padded.view(nb, BLOCK, kb, BLOCK).abs().amax(dim=(1, 3)) / E4M3_MAX
    q = w / scales.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(g, M, K).to(torch.bfloat16)
        if case["form"] == "linear":
            s["x"] = x
        else:
            s["xq"], s["x_scale"] = _quantised(x)
        s["wq"], s["w_scale"] = _block_weight(g, N, K)
        s["add"] = torch.randn((N,), generator=g, device=DEVICE) if case["bias"] else None
        return s
    M, H, I = case["M"], case["H"], case["I"]
    dt = DTYPES[case["dtype"]]
    if case["form"] == "fp8":
        s["x"] = _activations(g, M, H).to(dt)
        s["wq"], s["w_scale"] = _block_weight(g, 2 * I, H)
        return s
    # rows as a norm leaves them, weights that keep gate and up near one
    s["x"] = torch.randn((M, H), generator=g, device=DEVICE).to(dt)
    s["w"] = (torch.randn((2 * I, H), generator=g, device=DEVICE) / math.sqrt(H)).to(dt)
    if case["form"] == "step":
        s["dh"] = torch.randn((M, I), generator=g, device=DEVICE).to(dt)
    return s


# ------------------------------------------------------------------------------------------ plain forms


def _quantised(x):
    """(e4m3 codes [M][K], fp32 scales [M][K / 128 rounded up]): scale = amax / 448 of each 128 channels,
    the codes x / scale to nearest; a group of zeros has scale 0."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    padded = torch.zeros((M, kb * BLOCK), device=x.device)
    padded[:, :K] = x.float()
    groups = padded.view(M, kb, BLOCK)
    amax = groups.abs().amax(dim=2)
    scale = amax / torch.full_like(amax, E4M3_MAX)      # a true division: by a number it would be a product
    q = groups / torch.where(scale > 0, scale, 1.0)[:, :, None]
    q = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, kb * BLOCK)[:, :K].contiguous(), scale


def _rows(q, scale):
    """fp32 values of codes with one scale per row and 128 channels."""
    return q.float() * scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _blocks(q, scale):
    """fp32 values of codes with one scale per block of 128 x 128."""
    return _rows(q, scale.repeat_interleave(BLOCK, 0)[:q.shape[0]])


def _act(g, kind):
    """(act(g), act'(g))"""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    t = torch.tanh(GELU_C * (g + GELU_K * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_K * g * g)


def _plain(s):
    if s["op"] == "fp8":
        xq, xs = _quantised(s["x"]) if s["form"] == "linear" else (s["xq"], s["x_scale"])
        y = torch.matmul(_rows(xq, xs), _blocks(s["wq"], s["w_scale"]).t())
        if s["add"] is not None:
            y = y + s["add"]
        return {"y": y.to(DTYPES[s["out"]])}
    I, dt = s["I"], DTYPES[s["dtype"]]
    if s["form"] == "fp8":
        x, w = _rows(*_quantised(s["x"])), _blocks(s["wq"], s["w_scale"])
    else:
        x, w = s["x"].float(), s["w"].float()
    pre = torch.matmul(x, w.t())
    a, slope = _act(pre[:, :I], s["act"])
    out = {"h": (a * pre[:, I:]).to(dt)}
    if s["form"] == "step":
        dh = s["dh"].float()
        dpre = torch.cat([dh * pre[:, I:] * slope, dh * a], dim=1)
        out["dx"] = torch.matmul(dpre, w).to(dt)
        out["dw"] = torch.matmul(dpre.t(), x).to(dt)
    return out


# ----------------------------------------------------------------------------------- the framework's calls


def _own(s):
    import dequant_gemm_amd as cq

    if s["op"] == "fp8":
        weight = cq.Fp8Weight(s["wq"], s["w_scale"])
        if s["form"] == "linear":
            return {"y": cq.cubic_linear_fp8(s["x"], weight, bias=s["add"], out_dtype=DTYPES[s["out"]])}
        return {"y": cq.cubic_gemm_fp8(s["xq"], s["x_scale"], weight, bias=s["add"], out_dtype=DTYPES[s["out"]])}
    if s["form"] == "fp8":
        weight = cq.Fp8Weight(s["wq"], s["w_scale"])
        return {"h": cq.cubic_gated_ff_fp8(s["x"], weight, act=s["act"], out_dtype=DTYPES[s["dtype"]])}
    if s["form"] == "plain":
        return {"h": cq.cubic_gated_ff(s["x"], s["w"], act=s["act"])}
    h, pre = cq.cubic_gated_ff(s["x"], s["w"], act=s["act"], save_pre=True)
    dx, dw = cq.cubic_gated_ff_backward(s["dh"], s["x"], s["w"], pre, act=s["act"])
    return {"h": h, "dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work of one pass


def work(case):
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if case["op"] == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        read = M * K * 2 if case["form"] == "linear" else M * K + 4 * M * blocks(K)
        read += N * K + 4 * blocks(N) * blocks(K) + (4 * N if case["bias"] else 0)
        return {"bytes": read + M * N * (4 if case["out"] == "f32" else 2), "flops": 2.0 * M * N * K}
    M, H, I = case["M"], case["H"], case["I"]
    if case["form"] == "fp8":
        read = 2 * M * H + 2 * I * H + 4 * blocks(2 * I) * blocks(H)
        return {"bytes": read + 2 * M * I, "flops": 4.0 * M * H * I}
    if case["form"] == "plain":
        return {"bytes": 2 * (M * H + 2 * I * H + M * I), "flops": 4.0 * M * H * I}
    # x, w and dh in, h, dx and dw out: three products of the same size
    return {"bytes": 2 * (2 * M * H + 4 * I * H + 2 * M * I), "flops": 12.0 * M * H * I}


# ------------------------------------------------------------------- the definitions in 64 bits, for reference


def _exact_e4m3(v):
    """float64 values to the nearest e4m3 one, ties to even, by arithmetic: three fraction bits above 2^-6,
    steps of 2^-9 below."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(s):
    """float64 activations [M][K] as the quantised form has them."""
    if "xq" in s:
        q, scale = s["xq"].double(), s["x_scale"].double()
        return torch.cat([q[:, k * BLOCK:(k + 1) * BLOCK] * scale[:, k:k + 1] for k in range(scale.shape[1])], dim=1)
    parts = []
    for part in s["x"].float().split(BLOCK, dim=1):
        amax = part.abs().max(dim=1, keepdim=True)[0]
        # scale and quotient are fp32 by definition; 53 bits hold enough of a quotient to round it once more
        scale = (amax.double() / E4M3_MAX).float().double()
        quotient = (part.double() / torch.where(scale > 0, scale, 1.0)).float().double()
        parts.append(_exact_e4m3(quotient) * scale)
    return torch.cat(parts, dim=1)


def _exact_blocks(s):
    w = s["wq"].double()
    for n in range(s["w_scale"].shape[0]):
        for k in range(s["w_scale"].shape[1]):
            w[n * BLOCK:(n + 1) * BLOCK, k * BLOCK:(k + 1) * BLOCK] *= s["w_scale"][n, k].double()
    return w


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fp8":
        y = torch.einsum("mk,nk->mn", _exact_rows(s), _exact_blocks(s))
        return {"y": y if s["add"] is None else y + s["add"].double()[None, :]}
    I = case["I"]
    x, w = (_exact_rows(s), _exact_blocks(s)) if case["form"] == "fp8" else (s["x"].double(), s["w"].double())
    gate, up = torch.einsum("mk,nk->mn", x, w[:I]), torch.einsum("mk,nk->mn", x, w[I:])
    if case["act"] == "silu":
        p = torch.sigmoid(gate)
        value, slope = gate * p, p + gate * p * torch.sigmoid(-gate)
    else:  # 0.5 g (1 + tanh z) = g sigmoid(2 z)
        p = torch.sigmoid(2.0 * GELU_C * gate * (1.0 + GELU_K * gate.square()))
        value = gate * p
        slope = p + gate * p * (1.0 - p) * 2.0 * GELU_C * (1.0 + 3.0 * GELU_K * gate.square())
    out = {"h": value * up}
    if case["form"] == "step":
        dh = s["dh"].double()
        dgate, dup = dh * up * slope, dh * value
        out["dx"] = torch.einsum("mi,ih->mh", dgate, w[:I]) + torch.einsum("mi,ih->mh", dup, w[I:])
        out["dw"] = torch.cat([torch.einsum("mi,mh->ih", dgate, x), torch.einsum("mi,mh->ih", dup, x)], dim=0)
    return out
