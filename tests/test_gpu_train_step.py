"""The example training step: loss and imbalance fall under both ways of balancing, padding
takes no expert, and a step's gradients are those of its parts."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_step  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_example_trains_and_balances_by_the_loss():
    layer = train_step.Layer(T=1024, H=256, I=128, E=16, k=2)
    first, last = train_step.train(layer, steps=60, every=59, log=lambda *_: None)
    assert last[0] < 0.7 * first[0]
    # balance is 1 where shares and counts are even; uneven ones that oppose each other give less
    assert abs(last[1] - 1.0) < abs(first[1] - 1.0)


def test_example_trains_with_the_moving_bias():
    layer = train_step.Layer(T=1024, H=256, I=128, E=16, k=2)
    first, last = train_step.train(layer, steps=60, balance="bias", every=59, log=lambda *_: None)
    assert last[0] < 0.7 * first[0] and (layer.sel_bias != 0).any()


def test_the_moving_bias_evens_the_loads_of_a_fixed_router():
    from moe_expert_router_gb300 import binding as B
    layer = train_step.Layer(T=1024, H=256, I=128, E=16, k=2)
    loads = []
    with torch.no_grad():
        for _ in range(300):                             # 300 x 0.002 covers the scores' range
            _, _, r = layer.loss(0.0, 0.0)
            B.moe_bias_update(layer.sel_bias, r.counts, 0.002)
            c = r.counts.sum(0).double()
            loads.append((c.max() / c.mean()).item() - 1.0)
    assert loads[-1] < 0.5 * loads[0]


def test_padding_takes_no_expert_and_no_gradient():
    layer = train_step.Layer(T=512, H=128, I=64, E=8, k=2)
    layer.x = layer.x.clone().requires_grad_()
    loss, _, r = layer.loss(0.01, 1e-3)
    loss.backward()
    pad = ~layer.mask
    assert pad.any() and (r.topk_idx[pad] == -1).all() and (r.topk_w[pad] == 0).all()
    assert (layer.x.grad[pad] == 0).all() and (layer.x.grad[layer.mask].abs().sum(1) > 0).all()
    assert int(r.counts.sum()) == int(layer.mask.sum()) * layer.k
    assert all(torch.isfinite(p.grad).all() for p in layer.params)


def test_router_gradient_against_differences():
    """d loss / d w_r along a direction, through route, moe_experts and both terms, against the
    difference of the loss in the plain form in 64 bits on the same routing."""
    layer = train_step.Layer(T=256, H=128, I=64, E=8, k=2, seed=3)
    loss, _, r = layer.loss(0.5, 0.05)
    loss.backward()
    gen = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randn(layer.w_r.shape, generator=gen, device="cuda")
    got = (layer.w_r.grad.double() * d.double()).sum().item()

    x, w1, w2 = (t.detach().double() for t in (layer.x, layer.w1, layer.w2))
    live, idx = layer.mask, r.topk_idx.long().clamp(min=0)

    def plain(w_r):
        l = x @ w_r.t()
        s = torch.sigmoid(l)
        sk = s.gather(1, idx)
        w = sk / sk.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        for j in range(layer.k):
            h = torch.einsum("th,tih->ti", x, w1[idx[:, j]])
            g, u = h.chunk(2, 1)
            y += w[:, j:j + 1] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, w2[idx[:, j]])
        miss = ((y - layer.target.double()).square().mean(1) * live).sum() / live.sum()
        bal, share = 0.0, s / s.sum(1, keepdim=True)
        off = layer.seq_offsets.tolist()
        for b in range(2):
            inside = live.clone()
            inside[:off[b]] = False
            inside[off[b + 1]:] = False
            n = inside.sum()
            bal = bal + (layer.E * r.counts[b] / (layer.k * n) * share[inside].sum(0) / n).sum() / 2
        z = (torch.logsumexp(l, 1).square() * live).sum() / live.sum()
        return miss + 0.5 * bal + 0.05 * z
    h = 1e-5
    w_r = layer.w_r.detach().double()
    want = ((plain(w_r + h * d.double()) - plain(w_r - h * d.double())) / (2 * h)).item()
    # the expert path keeps bf16 activations: its gradient is held to 1e-2 by its own tests
    assert abs(got - want) <= 1e-2 * abs(want) + 1e-2 * layer.w_r.grad.norm().item()
    assert abs(loss.item() - plain(w_r).item()) <= 1e-2 * abs(loss.item())
