"""One training step of a small layer of experts, on the library's operators alone.

    python examples/moe_train_step.py [--steps 30]

The layer:  logits = router(x)                      FP32 router GEMM (BF16x3)
            each token goes to its top-k experts    rows sorted by expert, offsets on the device
            h_e = x W1_e^T, relu(h)^2, y_e = h W2_e^T    products grouped by expert
            shared expert z = x V^T                 8-bit product, scales per 128 values
            out = z + sum_k gate_k y_k
Loss: mean squared distance to a target.  The backward pass takes the grouped and 8-bit
gradients (dgrad and wgrad) and the router's; AdamW then updates FP32 master weights, with
8-bit moments, and writes the BF16 copies that the next step's products read.  No step
reads anything back to the host before the loss is printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_dense_projection_gb300 as dp  # noqa: E402


class MoELayer:
    def __init__(self, hidden=256, inner=512, experts=16, top_k=2, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, device=device, generator=g) / shape[-1] ** 0.5
        self.experts, self.top_k = experts, top_k
        self.router = normal(experts, hidden)                # FP32
        self.w1, self.w2 = normal(experts, inner, hidden), normal(experts, hidden, inner)
        self.shared = normal(hidden, hidden)
        self.masters = [self.router, self.w1, self.w2, self.shared]
        self.w1_16, self.w2_16, self.shared_16 = (w.bfloat16() for w in self.masters[1:])
        self.opt = dp.AdamW(self.masters, lr=2e-3, weight_decay=0.01, state_bits=8,
                            copies=[None, self.w1_16, self.w2_16, self.shared_16])

    def route(self, x):
        """Each token's experts and gates, and the (token, choice) pairs sorted by expert."""
        logits = dp.router_fwd(x.float(), self.router)
        top, choice = logits.topk(self.top_k, dim=1)
        gates = top.softmax(1)
        order = choice.flatten().argsort(stable=True)
        counts = torch.zeros(self.experts, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, choice.flatten(), torch.ones_like(order, dtype=torch.int32))
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=x.device)
        offsets[1:] = counts.cumsum(0)
        return choice, gates, order, offsets

    def forward_backward(self, x, target):
        """(loss, gradients in the order of ``masters``)."""
        T = x.shape[0]
        choice, gates, order, offsets = self.route(x)
        token = order // self.top_k
        rows = x[token]                                            # sorted by expert

        h = dp.dp_gemm_fwd_grouped(rows, self.w1_16, offsets)
        r = h.float().relu()
        a = (r * r).bfloat16()
        y = dp.dp_gemm_fwd_grouped(a, self.w2_16, offsets, out_dtype=torch.float32)

        xq, xs, xq_col, xs_col = dp.fp8_quantize(x, "both")       # forward and weight gradient, one read
        vq, vs = dp.fp8_quantize(self.shared_16, "block")
        out = dp.dp_gemm_fwd_fp8(xq, xs, vq, vs, out_dtype=torch.float32)
        gate = gates.flatten()[order]
        out.index_add_(0, token, y * gate[:, None])

        err = out - target
        loss = err.square().mean()
        d_out = err * (2.0 / err.numel())

        # shared expert
        dq, ds, dq_col, ds_col = dp.fp8_quantize(d_out, "both", dtype=torch.float8_e5m2)
        d_shared = dp.dp_gemm_wgrad_fp8(dq_col, ds_col, xq_col, xs_col, out_dtype=torch.float32)
        dx = dp.dp_gemm_dgrad_fp8(dq, ds, vq, vs, out_dtype=torch.float32)

        # experts
        d_rows = d_out[token]
        d_gate = (d_rows * y).sum(1)
        d_y = (d_rows * gate[:, None]).bfloat16()
        d_w2 = dp.dp_gemm_wgrad_grouped(d_y, a, offsets, out_dtype=torch.float32)
        d_a = dp.dp_gemm_dgrad_grouped(d_y, self.w2_16, offsets, out_dtype=torch.float32)
        d_h = (d_a * 2.0 * r).bfloat16()
        d_w1 = dp.dp_gemm_wgrad_grouped(d_h, rows, offsets, out_dtype=torch.float32)
        dx.index_add_(0, token, dp.dp_gemm_dgrad_grouped(d_h, self.w1_16, offsets, out_dtype=torch.float32))

        # router: the softmax of the chosen logits
        d_g = torch.empty_like(gates)
        d_g.view(-1)[order] = d_gate
        d_top = gates * (d_g - (d_g * gates).sum(1, keepdim=True))
        d_logits = torch.zeros(T, self.experts, device=x.device).scatter_(1, choice, d_top)
        d_router = dp.router_wgrad(d_logits, x.float())
        dx += dp.router_dgrad(d_logits, self.router)
        return loss, [d_router, d_w1, d_w2, d_shared], dx

    def step(self, x, target, max_norm=1.0):
        loss, grads, _ = self.forward_backward(x, target)
        norm = torch.stack([g.norm() for g in grads]).norm()
        clip = (max_norm / (norm + 1e-6)).clamp(max=1.0).reshape(1)  # stays on the device
        self.opt.step(grads, grad_scale=clip)
        return loss


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--tokens", type=int, default=2000)
    a = p.parse_args()
    layer, teacher = MoELayer(seed=0), MoELayer(seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    for i in range(a.steps):
        x = torch.randn(a.tokens, 256, device="cuda", generator=g).bfloat16()
        target = x.float() @ teacher.shared.T
        loss = layer.step(x, target)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}", flush=True)
    if dp.device_error():
        raise SystemExit("a kernel reported a timeout or wrong offsets")


if __name__ == "__main__":
    main()
