"""The trainable router at the edges of its definition: large finite masks among groups,
gradients that arrive at slots left over, NaN beside groups, near-ties behind ties, saturated
and vanishing scores, sums over many tokens. Against the formulas in 64 bits; tolerances as
in test_gpu_route.py where none is given."""
import numpy as np
import pytest
import torch

import route_reference as R
from moe_expert_router_gb300 import binding as B
from test_gpu_route import DEV, call, check, logits

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min
WIDTHS = [8, 24, 64, 128, 256, 512, 1024]                # every layout of lanes


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


@pytest.mark.parametrize("row,best", [
    ([50.0, 0.0, -1e4, 3.0, 20.0, 0.0, -1e4, -1e4], [0, 4]),
    ([0.0, 0.0, -1000.0, -30.0, -20.0, -20.0, -40.0, -40.0], [0, 1]),
    ([50.0, -1e4, LOWEST, 3.0, 20.0, LOWEST, LOWEST, LOWEST], [0, 4])])
def test_low_finite_logits_beside_a_group_at_the_border(row, best):
    l = torch.tensor([row], device=DEV)
    g, _ = check(l, 2, "softmax", n_group=4, topk_group=2, group_topn=2, backward=False)
    assert g["idx"][0].tolist() == best


@pytest.mark.parametrize("E,n_group", [(8, 4), (24, 4), (64, 16), (128, 8), (128, 32), (256, 16), (256, 32), (512, 32),
                                       (1024, 32)])
@pytest.mark.parametrize("mask", [-1e3, -1e4, LOWEST])
def test_groups_among_low_finite_logits(E, n_group, mask):
    """One expert far above the others, so that the sums of all other groups are within the error
    of 32-bit ones, and experts masked by a large finite number."""
    size = E // n_group
    rng = np.random.default_rng(E + n_group)
    l = rng.uniform(-30.0, 20.0, size=(60, E))
    l[rng.random((60, E)) < rng.choice([0.2, 0.6, 0.9], size=(60, 1))] = mask
    l[np.arange(60), rng.integers(0, E, 60)] = 50.0
    l[3, :size] = mask                                   # a group with nothing else
    l[5, 1:] = mask
    l = torch.tensor(l, dtype=torch.float32, device=DEV)
    for topn in (2, 3):
        if topn <= size:
            for stay in {2, n_group // 2}:
                check(l, min(6, stay * size), "softmax", n_group=n_group, topk_group=stay, group_topn=topn, backward=False)


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradients_at_slots_left_over_reach_nothing(E, score, normalize):
    """topk_w is the constant 0 there: infinity or NaN in its gradient (that of w log w, for one)
    leaves the row as it is."""
    rng = np.random.default_rng(E)
    T, k = 41, 6
    l = rng.normal(size=(T, E))
    for t in range(T):
        l[t, rng.permutation(E)[:E - 1 - t % k]] = -np.inf
    l[7] = -np.inf
    l = torch.tensor(l, dtype=torch.float32, device=DEV)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dlosses = torch.tensor([2.0, 0.5], device=DEV)
    clean = call(l, k, score, normalize, 1.5, dw=torch.tensor(dw, device=DEV), dlosses=dlosses)
    left = clean["idx"] < 0
    assert left.any() and torch.isfinite(clean["dl"]).all()
    for bad in (float("inf"), -float("inf"), float("nan")):
        d = torch.where(left, torch.tensor(bad, device=DEV), torch.tensor(dw, device=DEV))
        for losses, want in ((dlosses, clean), (None, None)):
            got = call(l, k, score, normalize, 1.5, dw=d, dlosses=losses)["dl"]
            if want is None:
                want = call(l, k, score, normalize, 1.5, dw=torch.tensor(dw, device=DEV))
            assert torch.equal(got, want["dl"])


@pytest.mark.parametrize("E,n_group", [(16, 2), (24, 4), (64, 8), (64, 2), (128, 4), (160, 8), (256, 8), (512, 4), (1024, 16)])
@pytest.mark.parametrize("topn", [2, 3])
@pytest.mark.parametrize("where", ["logit", "logit, a bias", "bias"])
def test_nan_takes_no_part_in_a_groups_sum(E, n_group, topn, where):
    """Group 0: a good expert, a NaN and poor ones; another group: two good ones a little lower."""
    size = E // n_group
    nan_at = {"logit": [1], "logit, a bias": [1, size - 1], "bias": [1]}[where]
    for other in (1, n_group - 1):
        l = torch.full((9, E), -5.0, device=DEV)
        l[:, 0] = 2.0
        l[:, other * size] = 1.5
        l[:, other * size + 1] = 1.375
        clean = l.clone()
        bias = None if where == "logit" else torch.full((E,), 0.25, device=DEV)
        if where == "bias":
            bias[1] = float("nan")
        else:
            l[4:, nan_at] = float("nan")
        g = call(l, 2, "sigmoid", n_group=n_group, topk_group=1, group_topn=topn, bias=bias)
        assert (g["idx"] == torch.tensor([other * size, other * size + 1], device=DEV)).all()
        # a NaN is as good as an expert that is off
        off = torch.where(torch.isnan(l), -float("inf"), clean)
        o = call(off, 2, "sigmoid", n_group=n_group, topk_group=1, group_topn=topn,
                 bias=None if bias is None else torch.where(torch.isnan(bias), -float("inf"), bias))
        assert torch.equal(o["idx"], g["idx"]) and torch.equal(o["w"], g["w"])


@pytest.mark.parametrize("E", [4, 8, 24, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_better_expert_behind_ties(E, dtype):
    """The first slots tie exactly (the same logit and bias), and an expert whose key equals theirs
    in 32 bits, but is larger, has a higher index."""
    for k in (1, 2, 8):
        if k + 2 > E:
            continue
        for last in (E - 1, k + 1):
            l = torch.full((21, E), -4.0, dtype=dtype, device=DEV)
            l[:, :k + 1] = 18.0
            l[::2, last] = 20.0                          # 1 - 2e-9 against 1 - 1.5e-8
            g, _ = check(l, k, "sigmoid", bias=torch.full((E,), 0.5, device=DEV), backward=False)
            assert g["idx"][0].tolist() == [last] + list(range(k - 1)) and g["idx"][1].tolist() == list(range(k))
            # softmax: scores of some 1e-13 under a bias of 1
            l = torch.full((21, E), -30.0, dtype=dtype, device=DEV)
            l[::2, last] = -29.0
            bias = torch.ones((E,), device=DEV)
            if last != k + 2 and k + 3 <= E:
                l[:, k + 2 if last == k + 1 else k + 1] = 0.0
                bias[k + 2 if last == k + 1 else k + 1] = -5.0
                # the selection alone: z is (log(1 + 4e-13))^2 here, below what 32 bits hold of 1 + 4e-13
                g = call(l, k, "softmax", bias=bias)
                r = R.route(l.double().cpu().numpy(), k, "softmax", bias=bias.cpu().numpy())
                assert np.array_equal(g["idx"].cpu().numpy(), r["idx"]) and g["idx"][0, 0] == last
                np.testing.assert_allclose(g["w"].cpu().numpy(), r["w"], rtol=1e-5)


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("steps", [1, 3])
def test_many_equal_logits_and_biases(E, steps):
    """Saturated bf16 logits of a few values under biases of a few values, as equal steps leave
    them: ties, and near-ties among them, without and with groups."""
    rng = np.random.default_rng(E * 10 + steps)
    l = torch.tensor(rng.integers(16, 22, size=(80, E)), dtype=torch.bfloat16, device=DEV)
    l[::3, E // 2:] = -3.0
    bias = torch.tensor(0.5 + rng.integers(0, steps, E) * 2.0 ** -23, dtype=torch.float32, device=DEV)
    for k in (1, 2, min(8, E // 2)):
        check(l, k, "sigmoid", bias=bias, backward=False)
        check(l, k, "sigmoid", bias=bias, n_group=4, topk_group=2, group_topn=2, backward=False)


def test_all_logits_equal_under_biases_of_two_values():
    for E in WIDTHS:
        bias = torch.where(torch.arange(E, device=DEV) % 3 == 1, 0.002, 0.001)
        g, _ = check(torch.zeros((33, E), device=DEV), 2, "sigmoid", bias=bias, backward=False)
        assert (g["idx"] == torch.tensor([1, 4], device=DEV)).all()


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_saturated_sigmoids(E, normalize):
    """s (1 - s) to a relative 2e-5 also where 1 - s is far below s's last digit: 1 - s = exp(-l) s
    carries exp's and s's errors, 2e-6 together; the rest is a sum held to its magnitudes."""
    rng = np.random.default_rng(E)
    T, k = 37, 3
    l = torch.tensor(rng.uniform(-25.0, 25.0, size=(T, E)), dtype=torch.float32, device=DEV)
    l[:9] = l[:9].abs() + 8.0
    l[9, 0], l[9, 1], l[9, 2] = 80.0, -80.0, 200.0
    dw = rng.normal(size=(T, k)).astype(np.float32)
    for dbal in (0.0, 4.0):
        g = call(l, k, "sigmoid", normalize, 1.5, dw=torch.tensor(dw, device=DEV), dlosses=torch.tensor([dbal, 0.0], device=DEV))
        ln = l.double().cpu().numpy()
        s, rest = 1.0 / (1.0 + np.exp(-ln)), 1.0 / (1.0 + np.exp(ln))
        r = R.route(ln, k, "sigmoid", normalize, 1.5)
        assert np.array_equal(g["idx"].cpu().numpy(), r["idx"])
        gs, size = np.zeros((T, E)), np.zeros((T, E))
        sk = np.take_along_axis(s, r["idx"], 1)
        base = sk.sum(1, keepdims=True) + 1e-20 if normalize else np.ones((T, 1))
        d = dw.astype(np.float64)
        cut = (d * sk).sum(1, keepdims=True) / base * normalize
        np.put_along_axis(gs, r["idx"], 1.5 / base * (d - cut), 1)
        np.put_along_axis(size, r["idx"], 1.5 / base * (np.abs(d) + (np.abs(d) * sk).sum(1, keepdims=True) / base * normalize), 1)
        a = dbal * E * r["counts"] / (k * float(T) ** 2)
        Z = s.sum(1, keepdims=True)
        gs += (a - (s * a).sum(1, keepdims=True) / Z) / Z
        size += (a + (s * a).sum(1, keepdims=True) / Z) / Z
        got = g["dl"].double().cpu().numpy()
        assert (np.abs(got - s * rest * gs) <= 2e-5 * s * rest * size + 1e-37).all()


@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("k", [1, 3])
def test_gradient_where_the_chosen_scores_vanish(E, k):
    """Chosen by their bias, with scores about the 1e-20 in the denominator: it has a gradient of
    its own, for a single weight and, through softmax, for the experts not chosen."""
    l = logits(43, E, seed=E, scale=0.5)
    l[:, E // 2] = torch.linspace(43.0, 52.0, 43, device=DEV)   # the others' scores: 3e-19 ... 3e-23
    bias = torch.full((E,), 3.0, device=DEV)
    bias[E // 2] = -3.0
    check(l, k, "softmax", bias=bias, scale=2.0)
    l[:, E // 2] = 1.0
    l -= torch.linspace(40.0, 52.0, 43, device=DEV)[:, None]
    check(l, k, "sigmoid", scale=2.0)


@pytest.mark.parametrize("row", [[1.0, 0.25, -0.5, 0.0], [2.0, 0.5, -1.0, 1.0]])
def test_sums_over_many_tokens(row):
    """134 million equal tokens: 64 additions in a row of a thread at most, 32 rows of a block, 26
    of the reduction, 2^-24 each, and a score's own error of 1e-6."""
    T, E = 1 << 27, 4
    l = torch.tensor(row, dtype=torch.bfloat16, device=DEV).repeat(T, 1)
    out = torch.empty((T, 1), dtype=torch.int32, device=DEV), torch.empty((T, 1), device=DEV)
    counts = torch.empty((1, E), dtype=torch.int32, device=DEV)
    tokens, losses = torch.empty((3,), dtype=torch.int32, device=DEV), torch.empty((2,), device=DEV)
    ws = torch.empty((B.moe_route_workspace_size(T, E, 1, 1),), dtype=torch.uint8, device=DEV)
    B.moe_route(l, B.router_cfg(), *out, counts=counts, seq_tokens=tokens, losses=losses, ws=ws)
    x = np.exp(np.array(row))
    assert counts[0].tolist() == [T, 0, 0, 0] and tokens.tolist() == [T, T, 1]
    want = np.array([E * x[0] / x.sum(), np.log(x.sum()) ** 2])
    np.testing.assert_allclose(losses.cpu().numpy(), want, rtol=(64 + 32 + 26) * 2.0 ** -24 + 2e-6)


@pytest.mark.parametrize("T,E,k", [(2_000_003, 8, 2), (200_001, 600, 4), (1_000_001, 100, 8)])
def test_sequences_longer_than_a_blocks_run(T, E, k):
    """Statistics of packed sequences whose part of a block is added in several runs, against the
    scores in 64 bits and the call's own indices; tolerances as above, and 4e-6 for a score's."""
    l = torch.randn((T, E), generator=torch.Generator(device=DEV).manual_seed(E), device=DEV).bfloat16()
    mask = torch.arange(T, device=DEV) % 7 != 3
    cuts = [0, T // 3, T // 3 + 1, T // 2, T // 2, T]
    offsets = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    S = len(cuts) - 1
    idx, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    counts = torch.empty((S, E), dtype=torch.int32, device=DEV)
    tokens, losses = torch.empty((S + 2,), dtype=torch.int32, device=DEV), torch.empty((2,), device=DEV)
    ws = torch.empty((B.moe_route_workspace_size(T, E, S, k),), dtype=torch.uint8, device=DEV)
    B.moe_route(l, B.router_cfg(), idx, w, token_mask=mask, seq_offsets=offsets, counts=counts, seq_tokens=tokens,
                losses=losses, ws=ws)
    balance, z, used = 0.0, 0.0, 0
    for b in range(S):
        rows = slice(cuts[b], cuts[b + 1])
        m = mask[rows]
        n = int(m.sum())
        assert torch.equal(counts[b], torch.bincount(idx[rows][m].flatten(), minlength=E).int()) and tokens[b] == n
        if n:
            x = l[rows][m].double()
            balance += (E * counts[b].double() / (k * n) * torch.softmax(x, 1).sum(0) / n).sum().item()
            z += torch.logsumexp(x, 1).square().sum().item()
            used += 1
    assert (idx[~mask] == -1).all() and tokens[S:].tolist() == [int(mask.sum()), used]
    want = np.array([balance / used, z / int(mask.sum())])
    np.testing.assert_allclose(losses.cpu().numpy(), want, rtol=(64 + 32 + 26) * 2.0 ** -24 + 4e-6)
