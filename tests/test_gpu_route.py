"""The trainable router's kernels against their formulas in 64 bits: selection (bit-exact
indices), weights, statistics, gradients; ties, near-ties, switched-off experts, padding,
packed sequences, strides and types.

Tolerances, from the roundings: a score's relative error is at most 5e-7 (sigmoid: exp 2 ulp,
an addition, a division) or 4e-6 (softmax: the rounding of l - max and a sum of up to 1024
terms); a normalised weight has it twice, so 1e-6 or 8e-6 plus a few 2^-24. Sums of n
positive terms add at most (additions in a row) 2^-24: 2e-5 covers them here. A gradient is
held to 2e-5 of the sum of the magnitudes that make it up, plus half a step of its type."""
import numpy as np
import pytest
import torch

import route_reference as R
from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import torch_ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
RTOL_W = {"sigmoid": 2e-6, "softmax": 1e-5}
RTOL_SUM = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def call(l, k, score="softmax", normalize=True, scale=1.0, n_group=1, topk_group=1, group_topn=1, bias=None, mask=None,
         offsets=None, dw=None, dlosses=None, stats=True):
    """The kernels' outputs on device tensors, as numpy."""
    T, E = l.shape
    S = 1 if offsets is None else len(offsets) - 1
    cfg = B.router_cfg(score, normalize, scale, n_group, topk_group, group_topn)
    out = dict(idx=torch.full((T, k), -7, dtype=torch.int32, device=DEV), w=torch.full((T, k), 99.0, device=DEV))
    kw = {}
    if stats:
        kw = dict(counts=torch.full((S, E), -7, dtype=torch.int32, device=DEV),
                  seq_tokens=torch.full((S + 2,), -7, dtype=torch.int32, device=DEV),
                  losses=torch.full((2,), 99.0, device=DEV))
    ws = torch.empty(B.moe_route_workspace_size(T, E, S, k), dtype=torch.uint8, device=DEV).fill_(0xff)
    B.moe_route(l, cfg, out["idx"], out["w"], sel_bias=bias, token_mask=mask, seq_offsets=offsets,
                ws=ws if stats else None, **kw)
    out.update(kw)
    if dw is not None:
        out["dl"] = torch.full((T, E), 99.0, dtype=l.dtype, device=DEV)
        B.moe_route_backward(l, cfg, out["idx"], dw, out["dl"], token_mask=mask, seq_offsets=offsets,
                             counts=kw.get("counts"), seq_tokens=kw.get("seq_tokens"), dlosses=dlosses)
    torch.cuda.synchronize()
    return out


def check(l, k, score="softmax", normalize=True, scale=1.0, n_group=1, topk_group=1, group_topn=1, bias=None, mask=None,
          offsets=None, backward=True, seed=0):
    T, E = l.shape
    rng = np.random.default_rng(seed)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dlosses = np.array([3.0 * T ** 0.5, 0.7 * T ** 0.5], np.float32)
    g = call(l, k, score, normalize, scale, n_group, topk_group, group_topn, bias, mask, offsets,
             torch.tensor(dw, device=DEV) if backward else None, torch.tensor(dlosses, device=DEV) if backward else None)
    ln = l.double().cpu().numpy()
    bn = None if bias is None else bias.cpu().numpy()
    mn = None if mask is None else mask.cpu().numpy() != 0
    on = None if offsets is None else offsets.cpu().numpy()
    r = R.route(ln, k, score, normalize, scale, n_group, topk_group, group_topn, bn, mn, on)
    assert np.array_equal(g["idx"].cpu().numpy(), r["idx"])
    assert np.array_equal(g["counts"].cpu().numpy(), r["counts"])
    assert np.array_equal(g["seq_tokens"].cpu().numpy(), r["seq_tokens"])
    np.testing.assert_allclose(g["w"].cpu().numpy(), r["w"], rtol=RTOL_W[score], atol=1e-37)
    np.testing.assert_allclose(g["losses"].cpu().numpy(), r["losses"].astype(np.float32), rtol=RTOL_SUM, atol=1e-30)
    if backward:
        want, size = R.route_backward(ln, r, dw.astype(np.float64), float(dlosses[0]), float(dlosses[1]), k, score, normalize, scale, on)
        eps = torch.finfo(l.dtype)
        bound = 2e-5 * size + 0.5 * eps.eps * np.abs(want) + 0.5 * float(eps.smallest_normal) * eps.eps + 1e-37
        got = g["dl"].double().cpu().numpy()
        assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / bound)
    # the same bits on every call, and the selection alone gives the same
    again = call(l, k, score, normalize, scale, n_group, topk_group, group_topn, bias, mask, offsets,
                 torch.tensor(dw, device=DEV) if backward else None, torch.tensor(dlosses, device=DEV) if backward else None)
    for name in g:
        assert torch.equal(g[name], again[name]), name
    alone = call(l, k, score, normalize, scale, n_group, topk_group, group_topn, bias, mask, None, stats=False)
    assert torch.equal(alone["idx"], g["idx"]) and torch.equal(alone["w"], g["w"])
    return g, r


def logits(T, E, dtype=torch.float32, seed=0, scale=1.0, pad=0, off=0):
    gen = torch.Generator().manual_seed(seed)
    full = (torch.randn((T, E + pad + off), generator=gen) * scale).to(dtype).to(DEV)
    return full[:, off:off + E]


@pytest.mark.parametrize("E,k", [(1, 1), (3, 3), (8, 2), (31, 32 - 1), (32, 32), (33, 4), (64, 6), (65, 7), (128, 8), (160, 6),
                                 (255, 8), (256, 32), (257, 5), (512, 9), (700, 10), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes(E, k, score):
    check(logits(37, E, seed=E), k, score, normalize=E % 2 == 0, scale=2.5, seed=E)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 31, 33, 300, 8000])
def test_token_counts(T):
    g, _ = check(logits(T, 48, seed=T), 4, "sigmoid", seed=T)
    if T == 0:
        assert g["losses"].tolist() == [0.0, 0.0] and int(g["counts"].sum()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (1, 0), (7, 3)])
@pytest.mark.parametrize("E", [24, 64, 104, 256])
def test_types_and_strides(dtype, pad, off, E):
    l = logits(61, E, dtype, seed=E + pad, pad=pad, off=off)
    bias = torch.randn((E,), generator=torch.Generator().manual_seed(1)).mul(0.05).to(DEV)
    check(l, 5, "sigmoid", bias=bias)


@pytest.mark.parametrize("E,n_group,topk_group,group_topn,k", [
    (8, 2, 1, 1, 3), (32, 32, 5, 1, 5), (64, 8, 4, 2, 8), (128, 4, 2, 1, 6), (160, 8, 3, 2, 6), (256, 8, 4, 2, 8),
    (256, 8, 8, 2, 8), (256, 16, 4, 16, 12), (512, 16, 4, 2, 8), (1024, 32, 4, 3, 16), (96, 3, 2, 4, 9), (1000, 8, 2, 5, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(E, n_group, topk_group, group_topn, k, score, with_bias):
    l = logits(50, E, torch.bfloat16, seed=E + k)
    l[7, : E // n_group] = -float("inf")                 # a group with nothing on
    l[9, : E - 2] = -float("inf")                        # only two experts on
    bias = torch.randn((E,), generator=torch.Generator().manual_seed(2)).mul(0.1).to(DEV) if with_bias else None
    check(l, k, score, n_group=n_group, topk_group=topk_group, group_topn=group_topn, bias=bias, scale=2.5)


@pytest.mark.parametrize("E", [8, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_index(E, with_bias):
    l = torch.zeros((19, E), device=DEV)
    l[3, 1::2] = -0.0                                    # the two zeros tie
    l[5, E // 2] = 1.0
    bias = torch.zeros((E,), device=DEV) if with_bias else None
    g, _ = check(l, 4, "sigmoid", bias=bias)
    assert g["idx"][0].tolist() == [0, 1, 2, 3] and g["idx"][5].tolist()[0] == E // 2
    check(l, 4, "softmax", n_group=2, topk_group=1, group_topn=1, bias=bias)


@pytest.mark.parametrize("E", [8, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_tie_in_32_bits_are_told_apart(E, score):
    """Scores whose difference is below fp32: the order is that of 64 bits."""
    rng = np.random.default_rng(E)
    if score == "sigmoid":
        l = torch.tensor(rng.uniform(17.0, 24.0, size=(40, E)), dtype=torch.float32, device=DEV)
        bias = torch.zeros((E,), device=DEV)
    else:                                                # bias differences of an ulp's size against small scores
        l = torch.tensor(rng.normal(size=(40, E)) * 1e-6, dtype=torch.float32, device=DEV)
        bias = torch.tensor(1.0 + rng.integers(0, 3, E) * 2.0 ** -23, dtype=torch.float32, device=DEV)
    check(l, 6, score, bias=bias, backward=False)
    check(l, 6 if E > 8 else 3, score, bias=bias, n_group=2, topk_group=1, group_topn=2, backward=False)


@pytest.mark.parametrize("E", [8, 20, 64, 128, 256, 300, 512, 1024])
@pytest.mark.parametrize("many", [False, True])
def test_saturated_scores_under_a_bias(E, many):
    """Sigmoid scores that are 1 in fp32 and a bias that is the same for all: the order is the
    logits', for a few experts of a row or all of them, with groups and without."""
    rng = np.random.default_rng(E)
    l = rng.normal(size=(60, E))
    for t in range(60):
        n = E if many else min(E, 1 + t % 7)
        l[t, rng.permutation(E)[:n]] = rng.uniform(17.0, 24.0, size=n)
    l[5, 0] = -np.inf
    l = torch.tensor(l, dtype=torch.float32, device=DEV)
    bias = torch.full((E,), 0.5, device=DEV)
    check(l, 4, "sigmoid", bias=bias, backward=False)
    if E % 4 == 0:
        check(l, 4, "sigmoid", bias=bias, n_group=4, topk_group=2, group_topn=1, backward=False)
        check(l, 3, "sigmoid", bias=bias, n_group=4, topk_group=2, group_topn=2, backward=False)
        check(l, 3, "sigmoid", n_group=4, topk_group=3, group_topn=2, backward=False)


@pytest.mark.parametrize("E", [8, 64, 256, 512])
@pytest.mark.parametrize("others", [0.0, 0.1])
def test_a_bias_of_minus_infinity_keeps_an_expert_out(E, others):
    l = logits(40, E, seed=E, scale=2.0)
    l[7] = 0.0                                           # ties
    bias = torch.full((E,), others, device=DEV)
    bias[1::2] = -float("inf")
    for kw in (dict(), dict(n_group=4, topk_group=2, group_topn=1), dict(n_group=4, topk_group=3, group_topn=2)):
        k = 4 if E > 8 else 3                            # fewer than k are left at E = 8 with groups
        for score in ("softmax", "sigmoid"):
            g, _ = check(l, k, score, bias=bias, **kw)
            assert not (g["idx"][g["idx"] >= 0] % 2 == 1).any()      # -1: left over
    bias[:] = -float("inf")
    g, _ = check(l, 3, "sigmoid", bias=bias)
    assert (g["idx"] == -1).all() and (g["w"] == 0).all()


@pytest.mark.parametrize("E,k", [(40, 20), (64, 31), (128, 17), (256, 24), (256, 32), (600, 30), (1024, 25)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_chosen_experts(E, k, dtype):
    """More chosen experts than a quarter of the lanes; bf16 logits tie often."""
    bias = torch.randn((E,), generator=torch.Generator().manual_seed(3)).mul(0.05).to(DEV)
    for b in (None, bias, bias.bfloat16().float()):
        check(logits(45, E, dtype, seed=E + k), k, "sigmoid", bias=b, backward=False)
        check(logits(45, E, dtype, seed=E + k, scale=3.0), k, "softmax", bias=b, n_group=2, topk_group=2, group_topn=2)


@pytest.mark.parametrize("E,k", [(16, 4), (64, 6), (128, 8), (256, 8), (1024, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_padding_off_experts_and_sequences(E, k, score):
    T = 210
    l = logits(T, E, seed=E)
    gen = torch.Generator().manual_seed(9)
    l[(torch.rand((T, E), generator=gen) < 0.3).to(DEV)] = -float("inf")
    l[20] = -float("inf")                                # nothing on
    l[30, 1:] = -float("inf")                            # fewer on than k
    l[40] = torch.finfo(torch.float32).min               # the type's lowest value everywhere is on
    mask = (torch.rand((T,), generator=gen) < 0.7).to(DEV)
    mask[20:60:10] = True
    mask[100:130] = False                                # a whole sequence of padding
    l[~mask] = float("nan")
    l[int((~mask).nonzero()[0])] = float("inf")
    for off in ([0, T], [0, 0, 1, 1, 100, 130, 131, 205, T], [0, T, T, T], list(range(T + 1))):
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        g, r = check(l, k, score, offsets=offsets, mask=mask, normalize=E != 64)
        dead = ~torch.tensor(r["live"], device=DEV)
        assert (g["idx"][dead] == -1).all() and (g["w"][dead] == 0).all() and (g["dl"][dead] == 0).all()
    check(l, k, score, mask=torch.zeros_like(mask))      # nothing live at all
    check(l, k, score, mask=mask.to(torch.uint8))


def test_lowest_values_and_extremes():
    l = torch.zeros((6, 16), device=DEV)
    l[0] = torch.linspace(-80, 80, 16)
    l[1] = -87.0
    l[1, 5] = -86.5
    l[2] = 88.0
    l[3, ::2] = torch.finfo(torch.float32).min
    l[4] = torch.linspace(-1e30, 1e30, 16)
    l[5, 3] = 200.0
    check(l, 3, "softmax", backward=False)
    check(l[:4], 3, "sigmoid")
    check(l[:4], 3, "softmax")


def test_nan_and_infinity_of_a_live_token():
    l = torch.randn((4, 32), generator=torch.Generator().manual_seed(0)).to(DEV)
    clean = call(l, 4, "softmax")
    l[1, 7] = float("nan")
    g = call(l, 4, "softmax")
    assert 7 not in g["idx"][1].tolist() and torch.isnan(g["w"][1]).all() and torch.isnan(g["losses"]).all()
    keep = [0, 2, 3]
    assert torch.equal(g["idx"][keep], clean["idx"][keep]) and torch.equal(g["w"][keep], clean["w"][keep])
    s = call(l, 4, "sigmoid")
    assert 7 not in s["idx"][1].tolist() and torch.isfinite(s["w"]).all()
    l[1, 7] = float("inf")
    s = call(l, 4, "sigmoid")
    assert s["idx"][1, 0] == 7 and torch.isfinite(s["w"]).all()


def test_nan_under_a_bias():
    l = torch.randn((3, 300), generator=torch.Generator().manual_seed(0)).to(DEV)
    bias = torch.full((300,), 0.25, device=DEV)
    bias[0] = 0.5
    clean = {score: call(l, 4, score, bias=bias) for score in ("softmax", "sigmoid")}
    l[1, 7] = float("nan")
    for score, c in clean.items():
        g = call(l, 4, score, bias=bias)
        assert torch.equal(g["idx"][[0, 2]], c["idx"][[0, 2]]) and torch.isnan(g["losses"]).all()
        if score == "softmax":                           # every key of the row is NaN
            assert (g["idx"][1] == -1).all() and (g["w"][1] == 0).all()
        else:
            assert 7 not in g["idx"][1].tolist() and (g["idx"][1] >= 0).all() and torch.isfinite(g["w"]).all()


def test_top1_normalised_weight_has_no_gradient():
    l = logits(77, 64, seed=4)
    dw = torch.randn((77, 1), generator=torch.Generator().manual_seed(1)).to(DEV)
    for score in ("softmax", "sigmoid"):
        g = call(l, 1, score, dw=dw, scale=2.5)
        assert (g["w"] == 2.5).all() and (g["dl"] == 0).all()


def test_backward_without_losses():
    l = logits(65, 40, seed=5)
    dw = torch.randn((65, 4), generator=torch.Generator().manual_seed(1)).to(DEV)
    for score in ("softmax", "sigmoid"):
        a = call(l, 4, score, dw=dw, normalize=False)
        b = call(l, 4, score, dw=dw, normalize=False, dlosses=torch.zeros((2,), device=DEV))
        assert torch.equal(a["dl"], b["dl"])


def test_offsets_past_32_bits():
    """Rows whose element offset passes 2^31 (a view of a 4.3 GB buffer)."""
    ld, E = 1 << 30, 64
    buf = torch.empty((2 * ld + E,), dtype=torch.bfloat16, device=DEV)
    l = torch.as_strided(buf, (3, E), (ld, 1))
    l.copy_(logits(3, E, torch.bfloat16, seed=8))
    check(l, 6, "softmax")


def test_many_tokens_and_long_sequences():
    T, E, k = 70001, 16, 2
    l = logits(T, E, torch.bfloat16, seed=11)
    offsets = torch.tensor([0, 3, 40000, 40000, T], dtype=torch.int32, device=DEV)
    check(l, k, "softmax", offsets=offsets)


def test_agrees_with_the_framework_router():
    """moe_route_logits on the same fp32 logits: the same experts (away from near-ties), weights
    and aux, which is the balance term of one softmax sequence without padding."""
    T, E, k = 500, 64, 6
    l = logits(T, E, seed=12).contiguous()
    shp = B.shape(T, 64, 64, E, k)
    ws = B.new_workspace(shp)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    aux = torch.zeros((1,), device=DEV)
    B.moe_route_logits(l, shp, B.router_cfg(), idx, w, ws, aux=aux)
    g = call(l, k)
    same = (g["idx"] == idx).all(1)
    assert same.float().mean() > 0.99
    torch.testing.assert_close(g["w"][same], w[same], rtol=2e-5, atol=0)
    torch.testing.assert_close(g["losses"][:1], aux, rtol=1e-4, atol=0)


def test_other_stream_and_graph_replay():
    T, E, k = 300, 128, 8
    l = logits(T, E, torch.bfloat16, seed=13)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
    dlosses = torch.tensor([2.0, 0.5], device=DEV)
    want = call(l, k, "sigmoid", dw=dw, dlosses=dlosses)
    cfg = B.router_cfg("sigmoid")
    out = {n: torch.zeros_like(t) for n, t in want.items()}
    ws = torch.empty(B.moe_route_workspace_size(T, E, 1), dtype=torch.uint8, device=DEV)

    def step():
        B.moe_route(l, cfg, out["idx"], out["w"], counts=out["counts"], seq_tokens=out["seq_tokens"], losses=out["losses"], ws=ws)
        B.moe_route_backward(l, cfg, out["idx"], dw, out["dl"], counts=out["counts"], seq_tokens=out["seq_tokens"],
                             dlosses=dlosses)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(out[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = logits(T, E, torch.bfloat16, seed=14)
    fresh = call(other, k, "sigmoid", dw=dw, dlosses=dlosses)
    l.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], fresh[n]) for n in fresh)


@pytest.mark.parametrize("L,S,E", [(1, 1, 1), (1, 1, 8), (3, 5, 33), (58, 7, 256), (2, 1000, 64), (2, 3, 1024)])
def test_bias_update(L, S, E):
    gen = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 4, (L, S, E), generator=gen, dtype=torch.int32).to(DEV)
    counts[0, 0] = 2 ** 31 - 1                           # sums past 32 bits
    bias = torch.randn((L, E), generator=gen).to(DEV)
    c = counts.long().sum(1).cpu()
    want = bias.cpu() + torch.sign(c.sum(1, keepdim=True) - E * c).float() * np.float32(0.01)
    B.moe_bias_update(bias, counts, 0.01)
    assert torch.equal(bias.cpu(), want)
    one = bias[0].clone()
    B.moe_bias_update(one, counts[0], 0.01)
    B.moe_bias_update(bias, counts, 0.01)
    assert torch.equal(one, bias[0])
    B.moe_bias_update(bias, counts[:, :0], 0.01)         # no sequences: no change
    assert torch.equal(one, bias[0])


def test_route_operator_under_autograd_and_compile():
    T, E, k = 150, 48, 4
    l = logits(T, E, torch.bfloat16, seed=15).contiguous()
    mask = torch.arange(T, device=DEV) % 9 != 0
    offsets = torch.tensor([0, 70, T], dtype=torch.int32, device=DEV)
    bias = torch.zeros((E,), device=DEV)
    weight = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)

    def f(l):
        r = torch_ops.route(l, k, "sigmoid", sel_bias=bias, token_mask=mask, seq_offsets=offsets)
        return (r.topk_w * weight).sum() + 0.3 * r.balance + 0.01 * r.z, r.topk_idx, r.counts
    grads = []
    for fn in (f, torch.compile(f, fullgraph=True, backend="aot_eager")):
        x = l.clone().requires_grad_(True)
        loss, idx, counts = fn(x)
        loss.backward()
        grads.append((loss.detach(), idx, counts, x.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    direct = call(l, k, "sigmoid", bias=bias, mask=mask, offsets=offsets, dw=weight,
                  dlosses=torch.tensor([0.3, 0.01], device=DEV))
    assert torch.equal(direct["dl"], grads[0][3]) and torch.equal(direct["idx"], grads[0][1])
    # only one of the outputs used, and logits whose experts are not consecutive
    x = l.t().contiguous().requires_grad_(True)
    torch_ops.route(x.t(), k, "softmax").z.backward()
    y = l.clone().requires_grad_(True)
    torch_ops.route(y, k, "softmax").z.backward()
    assert torch.equal(x.grad.t(), y.grad)


def test_experts_gradients_match_the_layer():
    """moe_experts on a routing equals the same step through moe_layer: y, dX without the router's
    term, dW1, dW2; and its routing-weight gradient is the library's."""
    T, H, I, E, k = 200, 128, 64, 8, 2
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=gen).bfloat16().to(DEV)
    w_r = (torch.randn((E, H), generator=gen) * 0.02).to(DEV)
    w1 = (torch.randn((E, 2 * I, H), generator=gen) * H ** -0.5).bfloat16().to(DEV)
    w2 = (torch.randn((E, H, I), generator=gen) * I ** -0.5).bfloat16().to(DEV)
    dy = torch.randn((T, H), generator=gen).bfloat16().to(DEV)
    a = [t.clone().requires_grad_(True) for t in (x, w_r, w1, w2)]
    y, idx, w, _ = torch_ops.moe_layer(*a, k)
    y.backward(dy)
    b = [t.clone().requires_grad_(True) for t in (x, w, w1, w2)]
    y2 = torch_ops.moe_experts(b[0], idx, b[1], b[2], b[3])
    y2.backward(dy)
    assert torch.equal(y, y2) and torch.equal(a[2].grad, b[2].grad) and torch.equal(a[3].grad, b[3].grad)
    import oracle
    ref = oracle.expert_backward(x, idx.cpu(), w.cpu().double(), w1, w2, dy)
    for got, want in ((b[1].grad, ref.dtopk_w), (b[0].grad, ref.dx)):
        g = got.float().cpu().double().numpy()
        assert np.linalg.norm(g - want) <= 1e-2 * np.linalg.norm(want)
    # dropped slots (padding): their rows get nothing, the others are unchanged
    idx3, w3 = idx.clone(), w.clone()
    idx3[10:20], w3[10:20] = -1, 0.0
    y3 = torch_ops.moe_experts(x, idx3, w3, w1, w2)
    assert (y3[10:20] == 0).all() and torch.equal(y3[20:], y[20:]) and torch.equal(y3[:10], y[:10])
