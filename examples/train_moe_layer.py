"""One MoE layer trained on one GPU with this library: router, dispatch, the
experts' feed-forward, combine, their backward passes, clipping and a plain
gradient step.  PyTorch holds the memory and computes the router's two small
products; everything else is the library's calls, in the order a training
program makes them.

    python examples/train_moe_layer.py [--steps 30]

Forward:   logits -> router_topk -> plan -> dispatch -> ffn -> combine
Backward:  combine_backward (down to the logits) -> ffn_backward ->
           combine with weights of 1 (the dispatch's backward pass)
Update:    clip_grad_norm over every gradient -> gradient step
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import combine_moe_dispatch_gb300 as moe


class MoELayer:
    """Parameters, gradients and the buffers of one batch size."""

    def __init__(self, tokens, hidden, intermediate, experts, top_k, capacity=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")

        def normal(*dims, std):
            return torch.empty(dims, **bf16).normal_(0.0, std, generator=g)

        self.I = intermediate
        self.shape = s = moe.make_shape(1, tokens, hidden, experts, top_k, capacity or tokens)
        self.w_router = normal(experts, hidden, std=hidden ** -0.5).float()
        self.w_gate_up = normal(experts, 2 * intermediate, hidden, std=hidden ** -0.5)
        self.w_down = normal(experts, hidden, intermediate, std=intermediate ** -0.5)
        self.params = [self.w_router, self.w_gate_up, self.w_down]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.b = moe.Buffers(s)
        # one workspace for the plan and the feed-forward
        self.b.workspace = torch.zeros(moe.ffn_workspace_size(s, intermediate), dtype=torch.uint8,
                                       device="cuda")
        self.clip_workspace = torch.zeros(moe.clip_workspace_size(), dtype=torch.uint8, device="cuda")
        self.topk_idx = torch.empty((tokens, top_k), dtype=torch.int32, device="cuda")
        self.topk_weights = torch.empty((tokens, top_k), device="cuda")
        self.ones = torch.ones((tokens, top_k), device="cuda")
        rows = (experts, s.capacity)
        self.expert_h = torch.empty((*rows, 2 * intermediate), **bf16)
        self.expert_act = torch.empty((*rows, intermediate), **bf16)
        self.d_expert_y = torch.empty((*rows, hidden), **bf16)
        self.d_expert_h = torch.empty((*rows, 2 * intermediate), **bf16)
        self.d_expert_x = torch.empty((*rows, hidden), **bf16)
        self.d_weights = torch.empty((tokens, top_k), device="cuda")
        self.d_logits = torch.empty((tokens, experts), device="cuda")
        self.d_x = torch.empty((tokens, hidden), **bf16)
        self.grad_norm = torch.zeros(1, device="cuda")

    def forward(self, x):
        s, b = self.shape, self.b
        self.x = x
        moe.router_topk(s, (x.float() @ self.w_router.t()).contiguous(), self.topk_idx, self.topk_weights)
        b.plan(self.topk_idx)
        b.dispatch(x, self.topk_idx)
        moe.ffn(s, self.I, b.expert_x, self.w_gate_up, self.w_down, b.expert_num_tokens, self.expert_h,
                self.expert_act, b.expert_y, b.workspace)
        b.combine(self.topk_idx, self.topk_weights)
        return b.y

    def backward(self, d_y):
        """Fills ``grads``; returns the gradient of x."""
        s, b = self.shape, self.b
        moe.combine_backward(s, d_y, b.expert_y, self.topk_idx, b.slot_of, self.topk_weights,
                             self.d_expert_y, self.d_weights, self.d_logits, b.workspace)
        moe.ffn_backward(s, self.I, self.d_expert_y, b.expert_x, self.expert_h, self.w_gate_up,
                         self.w_down, b.expert_num_tokens, self.expert_act, self.d_expert_h,
                         self.d_expert_x, self.grads[1], self.grads[2], b.workspace)
        # dispatch copied a token's row to its experts: their gradients add up
        moe.combine(s, self.d_expert_x, self.topk_idx, b.slot_of, self.ones, self.d_x, b.workspace)
        torch.mm(self.d_logits.t(), self.x.float(), out=self.grads[0])
        return self.d_x + (self.d_logits @ self.w_router).to(torch.bfloat16)

    def step(self, lr, max_norm):
        moe.clip_grad_norm(self.grads, self.grads, max_norm, self.grad_norm, self.clip_workspace)
        for p, g in zip(self.params, self.grads):
            p.add_(g, alpha=-lr)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    args = ap.parse_args()
    layer = MoELayer(tokens=512, hidden=512, intermediate=1024, experts=16, top_k=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((512, 512), device="cuda", generator=g).bfloat16()
    target = torch.randn((512, 512), device="cuda", generator=g)
    for i in range(args.steps):
        diff = layer.forward(x).float() - target
        layer.backward((diff / diff.shape[0]).bfloat16())
        layer.step(lr=0.5, max_norm=1.0)
        if i % 5 == 0 or i == args.steps - 1:
            print(f"step {i:3d}  loss {0.5 * float(diff.square().sum(1).mean()):9.4f}  "
                  f"gradient norm {float(layer.grad_norm):8.4f}")
    status = moe.read_status(layer.b.workspace)
    assert status == moe.Status.OK, status


if __name__ == "__main__":
    main()
