"""The optimizer's end of a step beside the rest of torch: writes that the tensors' version
counters show, constants in the host's digits, a step count for each parameter, and lists that
share memory."""
import numpy as np
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import optim, torch_ops
from moe_expert_router_gb300.mx_cache import MxWeightCache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def test_updates_move_the_version_counters():
    p, g = randn(40, 3, dtype=torch.bfloat16), randn(40, 3, seed=1, dtype=torch.bfloat16)
    o = optim.AdamW([p])
    before, read = p._version, g._version
    o.step([g], max_norm=1.0)
    assert p._version > before and g._version == read
    optim.grad_norm([g])
    assert g._version == read
    optim.clip_grad_norm_([g], 0.1)
    assert g._version > read
    bias, counts = torch.zeros((8,), device=DEV), torch.ones((1, 8), dtype=torch.int32, device=DEV)
    before = bias._version
    B.moe_bias_update(bias, counts, 0.1)
    assert bias._version > before
    with torch.inference_mode():                         # a tensor without a counter
        q = torch.ones((5,), device=DEV)
        optim.clip_grad_norm_([q], 0.5)
    optim.clip_grad_norm_([q], 0.25)
    assert abs(optim.grad_norm([q]).item() - 0.25) < 1e-5


def test_weight_copies_follow_an_update():
    w, g = randn(2, 4, 128, dtype=torch.bfloat16), randn(2, 4, 128, seed=1, dtype=torch.bfloat16)
    cache = MxWeightCache()
    old = [t.clone() for t in cache.get(w)]
    optim.AdamW([w], lr=0.5).step([g])
    new = cache.get(w)
    assert cache.quantizations == 2
    fresh = MxWeightCache().get(w)
    assert all(torch.equal(a, b) for a, b in zip(new, fresh)) and not torch.equal(new[0], old[0])


def test_a_backward_after_the_update_is_refused():
    T, H, I, E, k = 64, 128, 64, 4, 2
    x, w = randn(T, H, dtype=torch.bfloat16), torch.full((T, k), 0.5, device=DEV)
    w1 = (randn(E, 2 * I, H, seed=1) * H ** -0.5).bfloat16().requires_grad_()
    w2 = (randn(E, H, I, seed=2) * I ** -0.5).bfloat16().requires_grad_()
    idx = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k) % E
    y = torch_ops.moe_experts(x, idx, w, w1, w2)
    optim.AdamW([w1, w2], lr=0.1).step([torch.ones_like(w1), torch.ones_like(w2)])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()


def test_second_moment_at_the_default_betas():
    """v = (1 - b2) g^2 from nothing: 1 - 0.999 rounded once, two products, an addition of 0: four
    roundings of 2^-24. (With 1 - b2 taken from a rounded b2 it is off by 1.3e-5.)"""
    for betas in ((0.9, 0.999), (0.95, 0.9999)):
        p, g = randn(3000), randn(3000, seed=1)
        m, v = torch.zeros_like(p), torch.zeros_like(p)
        start = p.double().cpu().numpy()
        step, lr = torch.zeros((1,), dtype=torch.int32, device=DEV), torch.tensor([1e-3], device=DEV)
        optim.adamw_step([p], [g], [m], [v], step, lr, betas=betas, eps=1e-8, weight_decay=0.0)
        gn = g.double().cpu().numpy()
        np.testing.assert_allclose(v.double().cpu().numpy(), (1 - betas[1]) * gn ** 2, rtol=4 * 2.0 ** -24)
        np.testing.assert_allclose(m.double().cpu().numpy(), (1 - betas[0]) * gn, rtol=3 * 2.0 ** -24)
        # the first update is lr sign(g) (eps apart)
        want = -float(lr.item()) * gn / (np.abs(gn) + 1e-8)
        np.testing.assert_allclose(p.double().cpu().numpy() - start, want, rtol=5e-6, atol=2.0 ** -24 * np.abs(start).max())


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("bound", [0.0, 1.0])
def test_parameters_count_their_own_steps(skip, bound):
    """Against torch.optim.AdamW: a parameter whose gradient starts late, one whose gradient
    pauses, one that never has any, an empty one; with skipped steps between."""
    start = [randn(*s, seed=i) for i, s in enumerate(((33, 7), (1000,), (4,), (0,), (5,)))]
    ref = [s.clone().requires_grad_(True) for s in start]
    theirs = torch.optim.AdamW(ref, lr=0.01, weight_decay=0.1)
    ours = [s.clone().requires_grad_(True) for s in start]
    o = optim.AdamW(ours, lr=0.01, weight_decay=0.1, skip_nonfinite=skip)
    taken = 0
    for t in range(14):
        has = [True, t >= 6, t < 3 or t > 7, t != 1, False]
        for i, (a, b) in enumerate(zip(ref, ours)):
            a.grad = b.grad = None
            if has[i]:
                a.grad, b.grad = randn(*a.shape, seed=100 + 10 * t + i), randn(*a.shape, seed=100 + 10 * t + i)
        if skip and t in (2, 6, 8):
            ours[0].grad[1, 1] = float("nan")
        else:
            if bound:
                torch.nn.utils.clip_grad_norm_([a for a in ref if a.grad is not None], bound)
            theirs.step()
            taken += 1
        o.step(max_norm=bound)
        for a, b in zip(ref, ours):
            torch.testing.assert_close(b, a, rtol=2e-5, atol=2e-6)
    assert o.step_count.item() == taken and torch.equal(ours[4].detach(), start[4])


def test_own_step_counts_in_a_captured_step():
    """A captured step in which one parameter has no gradient, replayed, then an eager one of all."""
    start = [randn(300, seed=1), randn(70, seed=2)]
    ref = [s.clone().requires_grad_(True) for s in start]
    theirs = torch.optim.AdamW(ref, lr=0.01, weight_decay=0.0)
    o = optim.AdamW([s.clone() for s in start], lr=0.01, weight_decay=0.0)
    g = [randn(300, seed=3), randn(70, seed=4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o.step([g[0], None], 1e9)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o.step([g[0], None], 1e9)
    for _ in range(4):
        graph.replay()
    for t in range(8):
        ref[0].grad, ref[1].grad = g[0].clone(), g[1].clone() if t >= 5 else None
        theirs.step()
        if t >= 5:
            o.step(g, 1e9)
    for a, b in zip(ref, o.params):
        torch.testing.assert_close(b, a.detach(), rtol=2e-5, atol=2e-6)


def test_lists_that_share_memory_are_refused():
    """A tensor that a step writes may lie in no other of its lists."""
    n = 64
    buf = [randn(4 * n, seed=i) for i in range(5)]
    step, lr = torch.zeros((1,), dtype=torch.int32, device=DEV), torch.tensor([0.1], device=DEV)

    def lists():
        return [[b[:n], b[2 * n:3 * n]] for b in buf]
    before = [b.clone() for b in buf]
    for i in range(5):
        for j in range(5):
            if i == j:
                continue
            for at in (0, 1):
                for part in (lambda t, u: u, lambda t, u: buf[i][n - 1:2 * n - 1] if at == 0 else buf[i][3 * n - 1:4 * n - 1]):
                    a = lists()
                    a[j][at] = part(a[j][at], a[i][at])
                    p, g, m, v, x = a
                    with pytest.raises(ValueError, match="memory"):
                        optim.adamw_step(p, g, m, v, step, lr, masters=x)
    p, g, m, v, x = lists()
    for k in range(5):                                   # lr and step inside a list
        other = lists()
        other[k][0] = torch.zeros((n,), device=DEV)
        for bad in (dict(lr=other[k][0][3:4]), dict(step=other[k][0].view(torch.int32)[3:4])):
            if k == 1 and "lr" in bad:                   # both are only read
                continue
            with pytest.raises(ValueError, match="memory"):
                q = {**dict(step=step, lr=lr), **bad}
                optim.adamw_step(other[0], other[1], other[2], other[3], q["step"], q["lr"], masters=other[4])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(buf, before)) and step.item() == 0
    # neighbours, interleaved and out of order, are not shared
    whole = torch.zeros((10 * n,), device=DEV)
    cut = [whole[i * n:(i + 1) * n] for i in (7, 2, 9, 0, 4, 3, 8, 1, 6, 5)]
    optim.adamw_step(cut[:2], cut[2:4], cut[4:6], cut[6:8], step, lr, masters=[cut[8], cut[9]])
    optim.adamw_step(cut[:2], [g[0], g[0]], cut[4:6], cut[6:8], step, lr, masters=[None, cut[9]])   # a gradient read twice
    assert step.item() == 2


def test_a_restored_optimizer_goes_on():
    """Everything that a checkpoint holds, copied into a new AdamW: the next steps are the same."""
    start = [randn(300, seed=1).bfloat16(), randn(70, seed=2)]
    a = optim.AdamW([s.clone() for s in start], lr=0.01)
    for t in range(5):
        a.step([randn(300, seed=10 + t).bfloat16(), randn(70, seed=20 + t) if t > 2 else None], 1.0)
    b = optim.AdamW([p.clone() for p in a.params], lr=0.5)
    for x, y in ((a.exp_avg, b.exp_avg), (a.exp_avg_sq, b.exp_avg_sq), (a.masters, b.masters), ([a.step_count], [b.step_count]),
                 ([a.missed], [b.missed]), ([a.lr], [b.lr])):
        [v.copy_(u) for u, v in zip(x, y) if u is not None]
    for t in range(3):
        g = [randn(300, seed=30 + t).bfloat16(), randn(70, seed=40 + t)]
        a.step(g, 1.0)
        b.step(g, 1.0)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    assert a.missed.tolist() == [0, 3] and a.step_count.item() == 8
