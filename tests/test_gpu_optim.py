"""Gradient norm, clipping and AdamW over lists of tensors against their formulas in 64 bits.

Tolerances: the norm is summed in 64 bits from squares rounded in fp32 over 64 elements (at
most 18 roundings, 2^-24 each, halved by the root) and rounded once: 2e-6. A clipped element
is the factor's error (the norm's, an addition and a division: 3e-6) and its own product and
rounding. AdamW is some 20 fp32 operations, of which the division's argument m / (1 - b1^t)
carries the gradient's: 5e-6 of the magnitudes that make a value up, and half a step of its
type."""
import math

import numpy as np
import pytest
import torch

import route_reference as R
from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def tensors(sizes, dtypes=TYPES, scale=0.5, seed=0, odd=True):
    """Tensors of the sizes, each at an odd element of a buffer of its own where `odd`."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        at = (i * 3 + 1) % 9 if odd else 0
        buf = torch.empty((n + 9,), dtype=dtypes[i % len(dtypes)], device=DEV).normal_(0.0, scale, generator=gen)
        out.append(buf[at:at + n])
    return out


def values(ts):
    return [t.double().cpu().numpy() for t in ts]


LISTS = {"one element": [1], "empty ones": [0, 5, 0, 0, 3], "vector edges": list(range(1, 40)),
         "chunk edges": [16383, 16384, 16385, 32768, 4095, 4096, 4097, 3 * 16384 + 5], "one large": [3_000_001],
         "65": [17] * 65, "two tables": [11] * 1003, "blocks over": [20_000] * 64}


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("p", [1.0, 2.0, float("inf")])
def test_norm_and_clip(name, p):
    ts = tensors(LISTS[name], seed=len(name))
    before = values(ts)
    want = R.norm(before, p)
    got = optim.grad_norm(ts, p)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(got.item() - want) <= 2e-6 * want
    assert all(np.array_equal(a, b) for a, b in zip(before, values(ts)))
    # a bound above the norm changes nothing
    same = optim.clip_grad_norm_(ts, 2.0 * want, p)
    assert torch.equal(same, got) and all(np.array_equal(a, b) for a, b in zip(before, values(ts)))
    assert torch.equal(optim.clip_grad_norm_(ts, 0.25 * want, p), got)
    f = 0.25 * want / (want + 1e-6)
    for t, b, a in zip(ts, before, values(ts)):
        info = torch.finfo(t.dtype)
        assert (np.abs(a - b * f) <= (0.5 * info.eps + 4e-6) * np.abs(b * f) + info.smallest_normal * info.eps).all()


def test_neighbours_are_left_alone():
    buf = torch.full((40_000,), 3.0, dtype=torch.bfloat16, device=DEV)
    optim.clip_grad_norm_([buf[5:20_001], buf[20_003:39_990]], 1.0)
    assert (buf[:5] == 3).all() and (buf[20_001:20_003] == 3).all() and (buf[39_990:] == 3).all()
    assert (buf[5:20_001] < 3).all() and (buf[20_003:39_990] < 3).all()


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e-20, 1e-13, 1e13, 1e18, 1e25, 3e38])
def test_norm_over_the_whole_range(scale):
    """Squares that leave fp32, alone and next to ordinary values."""
    for n in (1, 700, 100_000):
        x = torch.full((n,), scale, device=DEV)
        y = torch.ones((n,), device=DEV)
        for ts in ([x], [x, y], [torch.cat([x, y])]):
            for p in (1.0, 2.0, float("inf")):
                want = R.norm(values(ts), p)
                if want > torch.finfo(torch.float32).max:
                    assert torch.isinf(optim.grad_norm(ts, p))
                else:
                    assert abs(optim.grad_norm(ts, p).item() - want) <= 2e-6 * want + 1.5e-45


def test_zeros_infinities_and_nan():
    z = [torch.zeros((5000,), device=DEV), torch.zeros((3,), dtype=torch.bfloat16, device=DEV)]
    for p in (1.0, 2.0, float("inf")):
        assert optim.clip_grad_norm_(z, 1.0, p).item() == 0.0 and all((t == 0).all() for t in z)
        for at in (0, 4321, 4999):
            for bad in (float("inf"), -float("inf"), float("nan")):
                ts = [torch.ones((5000,), device=DEV), torch.ones((9,), dtype=torch.float16, device=DEV)]
                ts[0][at] = bad
                n = optim.clip_grad_norm_(ts, 1.0, p)
                if math.isnan(bad):
                    assert torch.isnan(n) and all(torch.isnan(t).all() for t in ts)
                else:
                    assert torch.isinf(n) and torch.isnan(ts[0][at]) and (ts[1] == 0).all()
    assert optim.grad_norm([torch.empty((0,), device=DEV)]).item() == 0.0


def test_more_than_2_31_elements():
    x = torch.ones(((1 << 31) + 5,), dtype=torch.bfloat16, device=DEV)
    n = float(x.numel())
    assert abs(optim.grad_norm(x, 2.0).item() - math.sqrt(n)) <= 2e-6 * math.sqrt(n)
    optim.clip_grad_norm_(x, math.sqrt(n) / 2)
    assert (x == 0.5).all()


def test_dense_layouts_and_refusals():
    x = torch.randn((6, 5, 4), generator=torch.Generator().manual_seed(0)).to(DEV)
    n = optim.grad_norm([x.permute(2, 0, 1)])
    assert torch.equal(n, optim.grad_norm([x.contiguous()]))
    for bad in (x[:, ::2], x[:1].expand(6, 5, 4)):
        with pytest.raises(ValueError):
            optim.grad_norm([bad])
    with pytest.raises(TypeError):
        optim.grad_norm([x.double()])
    with pytest.raises(ValueError):
        optim.grad_norm([x], 3.0)
    with pytest.raises(ValueError):
        optim.grad_norm([x, x.cpu()])
    with pytest.raises(B.MoEError):
        optim.clip_grad_norm_([x], -1.0)
    y = x.clone()
    optim.clip_grad_norm_([y], 0.0)
    assert (y == 0).all()
    for shared in ([x, x], [x, x[5:]], [x[1:], x[:2]]):    # the same memory twice
        with pytest.raises(ValueError):
            optim.clip_grad_norm_(shared, 1.0)
    o = optim.AdamW([x])
    for g in (x.cpu(), x[:5], x.double(), x.permute(2, 0, 1).contiguous()):
        with pytest.raises((ValueError, TypeError)):
            o.step([g])
    with pytest.raises(TypeError):
        optim.adamw_step([x], [x], [x.half()], [x], o.step_count, o.lr)
    with pytest.raises(ValueError):
        optim.adamw_step([x.permute(2, 0, 1)], [x.permute(2, 0, 1).contiguous()], [x.permute(2, 0, 1)], [x.permute(2, 0, 1)],
                         o.step_count, o.lr)                # the same shape in another order of memory


CASES = {"fp32": (torch.float32, torch.float32, False), "bf16 with masters": (torch.bfloat16, torch.bfloat16, True),
         "bf16, fp32 gradients": (torch.bfloat16, torch.float32, True), "bf16 itself": (torch.bfloat16, torch.bfloat16, False),
         "fp16 with masters": (torch.float16, torch.float16, True)}


@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("sizes", [[1, 0, 7, 4096, 4097, 130_000], [33] * 70, [5] * 1200])
@pytest.mark.parametrize("odd", [False, True])
def test_adamw_steps(case, sizes, odd):
    pt, gt, with_master = CASES[case]
    ps = tensors(sizes, [pt], 0.5, 1, odd)
    ms, vs = tensors(sizes, [torch.float32], 0.01, 2, odd), tensors(sizes, [torch.float32], 0.01, 3, odd)
    [v.abs_() for v in vs]
    xs = [p.float() for p in ps] if with_master else None
    step, lr = torch.tensor([6], dtype=torch.int32, device=DEV), torch.tensor([0.01], device=DEV)
    b1, b2, eps, wd = 0.9, 0.95, 1e-8, 0.1
    # what the device holds of the fp32 constants
    c1, c2, ce, cw, cl = (float(np.float32(v)) for v in (b1, b2, eps, wd, 0.01))
    for t in (7, 8):
        gs = tensors(sizes, [gt], 0.3, 10 + t, odd)
        n = R.norm(values(gs), 2)
        most = 0.5 * n if t == 7 else 0.0
        old = [values(x) for x in (xs if with_master else ps, ms, vs)]
        norm = optim.adamw_step(ps, gs, ms, vs, step, lr, xs, (b1, b2), eps, wd, most)
        assert (norm is None) == (most == 0.0) and step.item() == t
        if norm is not None:
            assert abs(norm.item() - n) <= 2e-6 * n
        f = most / (n + 1e-6) if most else 1.0
        for i, g in enumerate(values(gs)):
            p, m, v = (o[i] for o in old)
            wp, wm, wv = R.adamw(p, g, m, v, t, cl, c1, c2, ce, cw, f)
            gp = (xs if with_master else ps)[i]
            half = 0.5 * torch.finfo(gp.dtype).eps
            u = np.abs(cl * (np.abs(m) + np.abs(g * f)) / (1 - c1 ** t) / (np.sqrt(wv / (1 - c2 ** t)) + ce))
            assert (np.abs(gp.double().cpu().numpy() - wp) <= (half + 5e-6) * np.abs(wp) + 5e-6 * (np.abs(p) + u) + 1e-30).all()
            assert (np.abs(ms[i].double().cpu().numpy() - wm) <= 5e-6 * (np.abs(m) + np.abs(g * f)) + 1e-38).all()
            assert (np.abs(vs[i].double().cpu().numpy() - wv) <= 1e-5 * wv + 1e-38).all()
            if with_master:
                assert torch.equal(ps[i], xs[i].to(pt))


def test_adamw_skips_a_step_that_is_not_finite():
    p, m, v = torch.ones((500,), device=DEV), torch.zeros((500,), device=DEV), torch.zeros((500,), device=DEV)
    g = torch.ones((500,), device=DEV)
    step, lr = torch.zeros((1,), dtype=torch.int32, device=DEV), torch.full((1,), 0.1, device=DEV)
    for bad in (float("inf"), float("nan")):
        g[77] = bad
        n = optim.adamw_step([p], [g], [m], [v], step, lr, skip_nonfinite=True)
        assert not torch.isfinite(n) and step.item() == 0 and (p == 1).all() and (m == 0).all() and (v == 0).all()
    g[77] = 1.0
    optim.adamw_step([p], [g], [m], [v], step, lr, skip_nonfinite=True)
    assert step.item() == 1 and (p < 1).all()


def test_optimizer_matches_torch_and_replays():
    """The class against torch.optim.AdamW in fp32 over ten steps, eager and as one captured
    step replayed, with a schedule written into lr and a parameter without a gradient."""
    gen = torch.Generator().manual_seed(0)
    start = [torch.randn(s, generator=gen).to(DEV) for s in ((33, 7), (1000,), (4,))]
    gs = [[torch.randn(s.shape, generator=gen).to(DEV) for s in start] for _ in range(10)]
    ref = [s.clone().requires_grad_(True) for s in start]
    theirs = torch.optim.AdamW(ref, lr=0.01, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    ours = [s.clone().requires_grad_(True) for s in start]
    o = optim.AdamW(ours, lr=0.01, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    held = [s.clone() for s in start]
    h = optim.AdamW(held, lr=0.01, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    static = [torch.zeros_like(s) for s in start[:2]]
    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in held + h.exp_avg + h.exp_avg_sq]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h.step(static + [None], 1.0)
    torch.cuda.current_stream().wait_stream(s)
    [a.copy_(b) for a, b in zip(held + h.exp_avg + h.exp_avg_sq, saved)]
    h.step_count.zero_()
    with torch.cuda.graph(graph):
        h.step(static + [None], 1.0)
    for t, g in enumerate(gs):
        rate = 0.01 / (1 + t)
        theirs.param_groups[0]["lr"] = rate
        o.lr.fill_(rate)
        h.lr.fill_(rate)
        for a, b, c in zip(ref[:2], ours[:2], g):
            a.grad, b.grad = c.clone(), c.clone()
        torch.nn.utils.clip_grad_norm_(ref[:2], 1.0)
        theirs.step()
        o.step(max_norm=1.0)
        [a.copy_(b) for a, b in zip(static, g)]
        graph.replay()
    for a, b, c in zip(ref, ours, held):
        torch.testing.assert_close(a, b, rtol=2e-5, atol=2e-6)
        assert torch.equal(b.detach(), c)
    assert torch.equal(ours[2].detach(), start[2])


def test_masters_follow_what_is_written_into_the_parameters():
    p = torch.randn((3, 40), generator=torch.Generator().manual_seed(0)).bfloat16().to(DEV)
    o = optim.AdamW([p], lr=0.0)
    p.fill_(2.0)
    o.refresh_masters()
    o.step([torch.ones_like(p)])
    assert (p == 2.0).all() and (o.masters[0] == 2.0).all()
