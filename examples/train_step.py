"""A training step of one MoE layer with balanced routing, clipping and AdamW.

    python examples/train_step.py [--steps 20] [--balance loss|bias]

The router's logits are a plain matrix product; selection, balance and z terms, the expert
path, their gradients, the clipping and the update run in libmoe. The batch is two packed
sequences with padding at their ends. With --balance loss the balance term joins the loss;
with --balance bias it is only watched, and the selection bias moves by the experts' counts
after every step. Nothing in a step waits for the device; the loss is read every few steps.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_expert_router_gb300 import binding as B  # noqa: E402
from moe_expert_router_gb300 import optim  # noqa: E402
from moe_expert_router_gb300.torch_ops import moe_experts, route  # noqa: E402


class Layer:
    """T tokens of width H through E experts of width I, k of them each."""

    def __init__(self, T=2048, H=512, I=256, E=32, k=4, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, scale=1.0, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=gen, device=device) * scale).to(dtype)
        self.E, self.k = E, k
        # tokens that lean towards few experts, so that there is something to balance
        self.x = randn(T, H) + 0.5 * randn(1, H)
        self.target = randn(T, H, scale=0.1)
        self.w_r = randn(E, H, scale=0.02, dtype=torch.float32).requires_grad_()
        self.w1 = randn(E, 2 * I, H, scale=H ** -0.5).requires_grad_()
        self.w2 = randn(E, H, I, scale=I ** -0.5).requires_grad_()
        self.sel_bias = torch.zeros((E,), device=device)
        split = T // 3
        self.seq_offsets = torch.tensor([0, split, T], dtype=torch.int32, device=device)
        self.mask = torch.ones((T,), dtype=torch.bool, device=device)
        self.mask[split - split // 8:split] = False          # padding
        self.mask[T - T // 16:] = False
        self.params = [self.w_r, self.w1, self.w2]

    def loss(self, balance_scale, z_scale):
        logits = self.x.float() @ self.w_r.t()
        r = route(logits, self.k, "sigmoid", sel_bias=self.sel_bias, token_mask=self.mask, seq_offsets=self.seq_offsets)
        y = moe_experts(self.x, r.topk_idx, r.topk_w, self.w1, self.w2)
        miss = ((y.float() - self.target).square().mean(1) * self.mask).sum() / self.mask.sum()
        return miss + balance_scale * r.balance + z_scale * r.z, miss.detach(), r


def train(layer, steps=20, balance="loss", lr=2e-3, max_norm=1.0, every=5, log=print):
    """Runs `steps` steps; returns the task loss and balance at the first and last."""
    opt = optim.AdamW(layer.params, lr=lr, betas=(0.9, 0.95), weight_decay=0.01, skip_nonfinite=True)
    seen = []
    for step in range(steps):
        for p in layer.params:
            p.grad = None
        loss, miss, r = layer.loss(0.01 if balance == "loss" else 0.0, 1e-5)
        loss.backward()
        norm = opt.step(max_norm=max_norm)
        if balance == "bias":
            B.moe_bias_update(layer.sel_bias, r.counts, 0.01)
        if step % every == 0 or step == steps - 1:
            seen.append((miss.item(), r.balance.item()))
            load = r.counts.sum(0).float()
            log(f"step {step:4d}  loss {miss.item():.5f}  balance {r.balance.item():.4f}  z {r.z.item():.3f}  "
                f"gradient norm {norm.item():.4f}  largest load {load.max().item() / load.mean().item():.2f} x mean")
    return seen[0], seen[-1]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--balance", choices=("loss", "bias"), default="loss")
    a = ap.parse_args()
    train(Layer(), a.steps, a.balance)
