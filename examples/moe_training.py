"""Training a mixture-of-experts feed-forward layer on one GPU, with its
activations kept in 8 bits until the backward pass.

    python examples/moe_training.py

    logits = x R^T                                  torch
    route  = the k best experts of every token      bsmm_route_topk
    h      = W_in,e x    for every (token, choice)  bsmm_expert_mm
    a, h8  = silu(h[:F]) * h[F:], h in 8 bits       bsmm_swiglu
    y      = weight * W_out,e a                     bsmm_expert_mm
    out    = sum of a token's y                     torch
    x8     = x in 8 bits                            bsmm_quant_int8_mx

and backward, from x8, h8 and the route alone:

    da      = W_out,e^T dout                        bsmm_expert_mm
    dh, weight * a, dweight                         bsmm_swiglu_backward
    dW_out  = sum of dout (weight * a)^T            bsmm_expert_wgrad
    dW_in   = sum of dh x8^T                        bsmm_expert_wgrad
    dx      = sum of W_in,e^T dh                    bsmm_expert_mm
    dlogits                                         bsmm_route_topk_backward
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_precision_gemm_amd as bsmm  # noqa: E402


class MoeLayer:
    """E experts of width F on D features, k per token; weights of ``dtype``,
    the router in fp32.  D and F are multiples of 32."""

    def __init__(self, D, F, E, k, *, alpha=0.01, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5

        self.k, self.alpha = k, alpha
        self.router = rand(E, D)
        self.w_in = rand(E, 2 * F, D).to(dtype)
        self.w_out = rand(E, D, F).to(dtype)

    def forward(self, x, mask=None):
        """x: [T, D].  Returns (out fp32 [T, D], the balance loss, what
        backward needs)."""
        T, D = x.shape
        logits = x.float() @ self.router.t()
        r = bsmm.bsmm_route_topk(logits, self.k, mask=mask, alpha=self.alpha)
        dt = x.dtype
        h = bsmm.bsmm_expert_mm(x, self.w_in, r.order, r.offsets, slots_per_row=self.k,
                                out_dtype=dt)
        a, h8, h_scale = bsmm.bsmm_swiglu(h, checkpoint=True)
        y = bsmm.bsmm_expert_mm(a, self.w_out, r.order, r.offsets, row_scale=r.weight.view(-1),
                                out_dtype="f32")
        x8, x_scale = bsmm.bsmm_quant_int8_mx(x)
        return y.view(T, self.k, D).sum(1), r.loss, (logits, r, mask, x8, x_scale, h8, h_scale)

    def backward(self, saved, dout):
        """dout: [T, D] of the layer's type.  Returns the gradients of x, the
        router, w_in and w_out for the task's loss plus the balance loss."""
        logits, r, mask, x8, x_scale, h8, h_scale = saved
        T, D = dout.shape
        k, dt = self.k, dout.dtype
        da = bsmm.bsmm_expert_mm(dout, self.w_out.transpose(1, 2), r.order, r.offsets,
                                 slots_per_row=k, out_dtype=dt)
        dh, a, dweight = bsmm.bsmm_swiglu_backward(da, h8, h_scale, row_scale=r.weight.view(-1))
        dw_out = bsmm.bsmm_expert_wgrad(dout, a, r.order, r.offsets, dy_slots_per_row=k)
        dw_in = bsmm.bsmm_expert_wgrad(dh, x8, r.order, r.offsets, x_scale=x_scale,
                                       x_slots_per_row=k)
        dx = bsmm.bsmm_expert_mm(dh, self.w_in.transpose(1, 2), r.order, r.offsets,
                                 out_dtype="f32").view(T, k, D).sum(1)
        dlogits = bsmm.bsmm_route_topk_backward(
            logits, r.index, r.weight, r.counts, r.live, dweight=dweight.view(T, k),
            dloss=torch.ones(1, device=dout.device), alpha=self.alpha, mask=mask)
        x = values(x8, x_scale)
        return dx + dlogits @ self.router, dlogits.t() @ x, dw_in, dw_out


def values(q, scale):
    """What an 8-bit checkpoint stands for, in fp32."""
    step = torch.exp2(scale.float() - 133)
    return q.float() * step.repeat_interleave(32, dim=1)


def main():
    torch.manual_seed(1)
    T, D, F, E, k = 2048, 1024, 512, 16, 4
    teacher, layer = MoeLayer(D, F, E, k, seed=1), MoeLayer(D, F, E, k, seed=2)
    layer.router.copy_(teacher.router)
    master = [layer.w_in.float(), layer.w_out.float()]
    for step in range(11):
        x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
        target, _, _ = teacher.forward(x)
        out, balance, saved = layer.forward(x)
        err = out - target
        if step % 5 == 0:
            kept = sum(t.numel() * t.element_size() for t in saved[3:])
            print(f"step {step}: task {err.square().sum(1).mean().item():.4f}, balance "
                  f"{balance.item():.4f}, activations kept {kept / 2**20:.1f} MiB", flush=True)
        _, d_router, d_in, d_out = layer.backward(saved, (2 * err / T).to(torch.bfloat16))
        layer.router -= 0.1 * d_router
        for p, g, w in zip(master, (d_in, d_out), (layer.w_in, layer.w_out)):
            p -= 20.0 * g
            w.copy_(p)


if __name__ == "__main__":
    main()
