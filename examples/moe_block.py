"""One routed-expert block, from the residual stream and back.

Serving: the residual's addition, the norm and its MXFP8 codes in one call
(kmoe_rmsnorm), the gate's logits (kmoe_router), group-limited routing
(kmoe_route_grouped) and the experts on the norm's codes (kmoe_forward_mx).

Tuning: the experts stay frozen MXFP4 weights; the gate learns.  The output's
gradient goes to the routing weights (kmoe_combine_backward, from the per-slot
outputs that the forward left in its workspace), to the logits
(kmoe_route_backward) and to the gate.  Through the gate it also reaches the
normed row, the norm's weight and the stream (kmoe_rmsnorm_backward), but that
is the router's share of their gradients only: the row acts on the output
through the experts too, and no call here gives that share (the experts'
weights are frozen, their dependence on the row is not).  So the norm's weight
is not stepped.  The target is the output of the same block under another gate,
so the loss can fall by routing alone.

    python examples/moe_block.py            # on a GB300
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp8_mxfp4_moe_gb300 as K  # noqa: E402
import workloads as W  # noqa: E402


class Block:
    """A block over T rows: a norm, a gate and frozen experts."""

    def __init__(self, w: W.Workload, n_group=4, topk_group=2, scale=2.5, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.w, self.route = w, dict(n_group=n_group, topk_group=topk_group, scale=scale)
        self.p = K.make_params(w.T, w.H, w.I, w.E, w.k)
        raw = W.gen_expert_weights_torch(w, "cuda")
        self.w13, self.w2 = K.kmoe_prepare_weights(self.p, raw["w13"], raw["w13_sf"], raw["w2"], raw["w2_sf"])
        self.gate = 0.05 * torch.randn(w.E, w.H, generator=g, device="cuda")
        self.norm = torch.ones(w.H, device="cuda")
        self.bias = 0.01 * torch.randn(w.E, generator=g, device="cuda")
        self.workspace = torch.empty(K.kmoe_workspace_size(self.p), dtype=torch.uint8, device="cuda")

    def forward(self, x, residual):
        """The block's output and what the backward pass needs."""
        h, y, codes, scales = K.kmoe_rmsnorm(x, self.norm, residual=residual, mx=True)
        logits = K.kmoe_router(y, self.gate.to(torch.bfloat16), self.bias, self.w.k)[2]
        ids, tw = K.kmoe_route_grouped(logits, self.bias, self.w.k, **self.route)
        out, ws = K.kmoe_forward_mx(self.p, codes, scales, ids, tw, self.w13, self.w2, workspace=self.workspace)
        return out, (h, y, logits, ids)

    def backward(self, d_out, saved):
        """The gate's gradient, and what reaches the norm's weight and the
        stream through the router: their gradients without the experts' share.
        The stream that goes on is h + out, so d_out is h's gradient too."""
        h, y, logits, ids = saved
        slots = K.stage_views(self.p, self.workspace)["y"]
        d_w = K.kmoe_combine_backward(d_out, slots, ids, self.w.E)
        d_logits = K.kmoe_route_backward(d_w, logits, ids, scale=self.route["scale"])
        d_gate = d_logits.t() @ y.float()
        dy = (d_logits @ self.gate).to(torch.bfloat16)
        d_h, d_norm = K.kmoe_rmsnorm_backward(dy, h, self.norm, dh_in=d_out)
        return d_gate, d_norm, d_h


def main(steps=20, rate=0.02):
    w = W.Workload("block", T=256, H=512, I=256, E=32, k=4)
    block = Block(w)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(w.T, w.H, generator=g, device="cuda").to(torch.bfloat16)
    residual = torch.randn(w.T, w.H, generator=g, device="cuda").to(torch.bfloat16)
    own = block.gate.clone()
    block.gate += 0.02 * torch.randn(w.E, w.H, generator=g, device="cuda")
    target = block.forward(x, residual)[0].float()
    block.gate = own
    losses = []
    for step in range(steps):
        out, saved = block.forward(x, residual)
        diff = (out.float() - target) / target.norm()
        losses.append(float(diff.square().sum()))
        d_gate, _, _ = block.backward(diff.to(torch.bfloat16), saved)
        # steps of one size, whatever the gradient's
        block.gate -= rate * block.gate.norm() * d_gate / d_gate.norm()
    st, word = K.kmoe_device_error(block.workspace)
    assert st == 0, f"device error {word:#x}"
    print(f"relative squared error: {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    return losses


if __name__ == "__main__":
    main()
