"""A mixture-of-experts feed-forward layer with 4-bit weights on one GPU.

    python examples/moe_layer.py

Quantises a shared expert and E routed experts, runs the layer on a batch of
tokens and on a single one, and trains the router for a few steps on the
task's gradient and the balance loss with the expert weights frozen:

    logits = x R^T                              torch
    route  = the k best experts of every token  bsmm_route_topk
    h      = W_in,e x  for every (token, choice)  bsmm_w4_expert_mm
    a      = silu(h[:F]) * h[F:]                torch
    y      = weight * W_out,e a                 bsmm_w4_expert_mm
    out    = sum of a token's y + shared expert  torch, bsmm_w4_mm
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_precision_gemm_amd as bsmm  # noqa: E402


def gate(h):
    """silu(first half) * second half, in fp32."""
    a, b = h.float().chunk(2, -1)
    return torch.nn.functional.silu(a) * b


class MoeLayer:
    """E experts of width F on D features, k per token, and one shared
    expert; weights in 4 bits, the router in fp32."""

    def __init__(self, D, F, E, k, *, group=128, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5

        def w4(w):
            q, scale, zero, values = bsmm.bsmm_quant_w4(w, group=group, symmetric=False,
                                                        scale_dtype="bf16", values=True)
            return (q, scale, zero), values

        self.E, self.k = E, k
        self.router = rand(E, D)
        # (operands, the values they stand for)
        self.w_in, self.w_in_values = w4(rand(E, 2 * F, D))
        self.w_out, self.w_out_values = w4(rand(E, D, F))
        self.s_in, self.s_in_values = w4(rand(2 * F, D))
        self.s_out, self.s_out_values = w4(rand(D, F))

    def __call__(self, x, *, mask=None, alpha=None):
        """x: bf16 [T, D].  Returns (out fp32 [T, D], what backward needs)."""
        T, D = x.shape
        logits = x.float() @ self.router.t()
        r = bsmm.bsmm_route_topk(logits, self.k, mask=mask, alpha=alpha)
        h = bsmm.bsmm_w4_expert_mm(x, *self.w_in, r.order, r.offsets, slots_per_row=self.k)
        # unweighted rows where a gradient of the weights is wanted
        y = bsmm.bsmm_w4_expert_mm(gate(h).to(x.dtype), *self.w_out, r.order, r.offsets,
                                   row_scale=None if alpha is not None else r.weight.view(-1),
                                   out_dtype="f32").view(T, self.k, D)
        routed = (y * r.weight[..., None]).sum(1) if alpha is not None else y.sum(1)
        shared = bsmm.bsmm_w4_mm(gate(bsmm.bsmm_w4_mm(x, *self.s_in)).to(x.dtype), *self.s_out,
                                 out_dtype="f32")
        return routed + shared, (x, logits, r, y, mask, alpha)

    def router_gradient(self, saved, dout):
        """Gradient of (task loss + balance loss) for the router, from the
        task's gradient of the output."""
        x, logits, r, y, mask, alpha = saved
        dweight = (y * dout[:, None]).sum(-1)
        dlogits = bsmm.bsmm_route_topk_backward(
            logits, r.index, r.weight, r.counts, r.live, dweight=dweight,
            dloss=torch.ones(1, device=x.device), alpha=alpha, mask=mask)
        return dlogits.t() @ x.float()


def main():
    torch.manual_seed(1)
    T, D, F, E, k = 512, 1024, 512, 16, 4
    layer = MoeLayer(D, F, E, k)
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    mask = torch.arange(T, device="cuda") < T - 12            # padding at the end
    target, _ = layer(x, mask=mask)
    layer.router += 0.3 * torch.randn_like(layer.router) / D ** 0.5     # to be learned back
    for step in range(21):
        out, saved = layer(x, mask=mask, alpha=0.5)
        err = (out - target) * mask[:, None]
        if step % 5 == 0:
            r = saved[2]
            print(f"step {step}: task {err.square().sum(1).mean().item():.4f}, balance "
                  f"{r.loss.item():.4f}, loads {int(r.counts.min())}..{int(r.counts.max())}",
                  flush=True)
        layer.router -= 0.002 * layer.router_gradient(saved, 2 * err / T)
    one, _ = layer(x[:1])
    batch, _ = layer(x, mask=mask)
    print(f"one token against the batch: {(one[0] - batch[0]).abs().max().item():.2e} of "
          f"{batch[0].abs().max().item():.2e}")


if __name__ == "__main__":
    main()
