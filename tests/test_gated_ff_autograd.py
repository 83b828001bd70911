"""The gated block beside autograd: it records no graph and says so, and the two calls make a differentiable function."""
import pytest
import torch

import dequant_gemm_amd as cq


def test_inputs_that_require_a_gradient_are_refused():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((64, 64), dtype=torch.bfloat16)
    for a, b in ((x.clone().requires_grad_(), w), (x, torch.nn.Parameter(w))):
        with pytest.raises(RuntimeError, match="no graph"):
            cq.cubic_gated_ff(a, b)
        with torch.no_grad(), pytest.raises(ValueError):          # what follows is the next check: a host tensor
            cq.cubic_gated_ff(a, b)


class _Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, act):
        h, pre = cq.cubic_gated_ff(x, w, act=act, save_pre=True)
        ctx.save_for_backward(x, w, pre)
        ctx.act = act
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w, pre = ctx.saved_tensors
        dx, dw = cq.cubic_gated_ff_backward(dh.contiguous(), x, w, pre, act=ctx.act, need_dx=ctx.needs_input_grad[0],
                                            need_dw=ctx.needs_input_grad[1])
        return dx, dw, None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 90])
def test_in_an_autograd_function(M, dtype):
    print(f"[gpu-case] gated_ff in an autograd function M={M} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w, dh = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((M, 128), (80, 128), (M, 40)))
    with torch.no_grad():
        parameter = torch.nn.Parameter(w)
        h, pre = cq.cubic_gated_ff(x, parameter, save_pre=True)   # without a graph a parameter is a tensor
    dx, dw = cq.cubic_gated_ff_backward(dh, x, w, pre)
    for need_x, need_w in ((True, True), (True, False), (False, True)):
        a, b = x.clone().requires_grad_(need_x), w.clone().requires_grad_(need_w)
        y = _Block.apply(a, b, "silu")
        assert torch.equal(y, h)
        y.backward(dh)
        assert (a.grad is None) == (not need_x) and (b.grad is None) == (not need_w)
        assert not need_x or torch.equal(a.grad, dx)
        assert not need_w or torch.equal(b.grad, dw)
