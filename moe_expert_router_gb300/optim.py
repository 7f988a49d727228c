"""The optimizer's end of a training step: gradient norm, clipping and AdamW over all
parameters at once, on libmoe's kernels.

The parameters and gradients that a call changes in place have their version counters moved, as
by torch's own optimizers: a backward through weights that a step has changed is refused, and an `MxWeightCache` quantizes
them again. A replayed graph moves no counter: call the cache's `invalidate()` beside it.

Every call takes whole lists of tensors (fp32, bf16, fp16, mixed; any sizes), enqueues
one or two kernels on the current stream (more for a list of many hundred tensors) and
reads nothing back: the norm, the clip
factor, the learning rate and the step count stay on the device, so a step can be
captured into a CUDA graph and replayed.
"""
from __future__ import annotations

import torch

from . import binding as B


def _lists(tensors, name):
    if isinstance(tensors, torch.Tensor):
        return [tensors]
    tensors = tensors if isinstance(tensors, (list, tuple)) else list(tensors)
    if not tensors:
        raise ValueError(f"{name} is empty")
    return tensors


def grad_norm(grads, norm_type=2.0):
    """The norm (norm_type 1, 2 or inf) of all elements of `grads` together, an fp32 scalar
    tensor on their device."""
    grads = _lists(grads, "grads")
    ws, norm = B.tensors_scratch(len(grads), grads[0])
    B.moe_grad_norm(grads, norm, ws, norm_type)
    return norm


def clip_grad_norm_(grads, max_norm, norm_type=2.0):
    """Multiplies every tensor of `grads` in place by min(1, max_norm / (norm + 1e-6)) and
    returns the norm before that, as a tensor on the device."""
    grads = _lists(grads, "grads")
    ws, norm = B.tensors_scratch(len(grads), grads[0])
    B.moe_clip_grads(grads, max_norm, norm, ws, norm_type)
    return norm


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr, masters=None, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=0.01, max_norm=0.0, skip_nonfinite=False, missed=None):
    """One AdamW step on tensors that the caller holds, in place. step int32 [1] and lr fp32 [1]
    are on the device; exp_avg, exp_avg_sq and masters fp32. With max_norm > 0 the gradients are
    taken times min(1, max_norm / (their global 2-norm + 1e-6)), without being changed. missed
    int32 [n] on the device: how many of the steps each parameter had no part in. Returns the norm as a tensor (None where max_norm is 0 and skip_nonfinite is False)."""
    params, grads = _lists(params, "params"), _lists(grads, "grads")
    ws, norm = B.tensors_scratch(len(params), params[0])
    if not (max_norm > 0.0 or skip_nonfinite):
        norm = None
    cfg = B.AdamWCfg(betas[0], betas[1], eps, weight_decay, max_norm, int(bool(skip_nonfinite)))
    B.moe_adamw(params, grads, exp_avg, exp_avg_sq, lr, step, ws, cfg, masters, norm, missed=missed)
    return norm


class AdamW:
    """AdamW over `params` with fp32 state, and fp32 masters for 16-bit parameters (masters=False:
    those are updated themselves, rounded to nearest at every step).

    `step(grads=None, max_norm=0.0)` uses the parameters' .grad where no list is given; parameters
    without a gradient are left alone, and their bias corrections go by the steps that they took
    part in: `step_count` less their `missed`. Those and `lr` are device tensors: write into `lr`
    for a schedule. `max_norm` bounds the norm of this step's gradients: parameters that are to be
    clipped together belong to one AdamW. What a checkpoint has to hold are `exp_avg`, `exp_avg_sq`,
    `masters`, `step_count`, `missed` and `lr`: copy into them (there is no state_dict). Masters are copies made here (`refresh_masters`)."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, masters=True,
                 skip_nonfinite=False):
        self.params = list(_lists(params, "params"))
        device = self.params[0].device
        self.betas, self.eps, self.weight_decay, self.skip_nonfinite = betas, eps, weight_decay, skip_nonfinite
        self.lr = torch.full((1,), lr, dtype=torch.float32, device=device)
        self.step_count = torch.zeros((1,), dtype=torch.int32, device=device)
        self.missed = torch.zeros((len(self.params),), dtype=torch.int32, device=device)
        self.exp_avg = [torch.zeros_like(p, dtype=torch.float32) for p in self.params]
        self.exp_avg_sq = [torch.zeros_like(p, dtype=torch.float32) for p in self.params]
        self.masters = [p.detach().float() if masters and p.dtype != torch.float32 else None for p in self.params]

    def refresh_masters(self):
        """Takes the masters from the parameters again, after something else wrote into those (a
        checkpoint that was loaded); a step writes the parameters from them."""
        for p, x in zip(self.params, self.masters):
            if x is not None:
                x.copy_(p.detach())

    def step(self, grads=None, max_norm=0.0):
        """One update; returns the gradients' norm as in adamw_step."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError("one gradient for each parameter")
        at = [i for i, g in enumerate(grads) if g is not None]
        if not at:
            return None
        part = len(at) < len(grads)
        missed = torch.cat([self.missed[i:i + 1] for i in at]) if part else self.missed
        before = self.step_count.clone() if part else None
        norm = adamw_step([self.params[i] for i in at], [grads[i] for i in at],
                          [self.exp_avg[i] for i in at], [self.exp_avg_sq[i] for i in at], self.step_count, self.lr,
                          [self.masters[i] for i in at], self.betas, self.eps, self.weight_decay, max_norm,
                          self.skip_nonfinite, missed)
        if part:
            taken = self.step_count - before             # 0 where the step was skipped
            for i, g in enumerate(grads):
                if g is None:
                    self.missed[i:i + 1].add_(taken)
        return norm
