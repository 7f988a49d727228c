"""Cases of the trainable router and of the optimizer end of a training step.

Four operators: the router's selection from logits with its balance terms (`route`,
forward alone as serving calls it, or forward and backward as training does), the update
of the selection bias from the experts' counts (`bias`), the global gradient norm with
clipping (`clip`), and the AdamW step that takes the clip factor on the device (`adamw`).

`run` computes them in elementary torch operations, or, where `own` is true, through this
repository's package.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _route(name, T, E, k, score, dtype, **more):
    case = dict(op="route", T=T, E=E, k=k, score=score, dtype=dtype, normalize=True, scale=1.0, n_group=1,
                topk_group=1, group_topn=1, bias=False, S=1, pad=0, masked=False, off=False, train=True)
    case.update(more)
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # serving, one token through a 256-expert router with groups and a selection bias: latency only
        _route("route one token", 1, 256, 8, "sigmoid", "f32", scale=2.5, n_group=8, topk_group=4, group_topn=2,
               bias=True, train=False),
        # a prompt through the 64-expert softmax router, logits as a bf16 router layer gives them
        _route("route prompt", 4096, 64, 6, "softmax", "bf16", train=False),
        # the training step's routing at 8192 tokens and 256 experts in groups, four packed sequences with padding
        _route("route train groups", 8192, 256, 8, "sigmoid", "f32", scale=2.5, n_group=8, topk_group=4,
               group_topn=2, bias=True, S=4, masked=True),
        # ragged sizes: groups of 20 experts, plain (unnormalised) weights, rows wider than the experts, switched-off experts
        _route("route train ragged", 5003, 160, 6, "softmax", "f16", normalize=False, scale=16.0, n_group=8,
               topk_group=3, group_topn=1, S=11, pad=7, masked=True, off=True),
        # the longest batch: many packed sequences of unlike lengths, popular and rare experts
        _route("route train long", 131072, 128, 8, "softmax", "bf16", S=37),
        # one layer's bias after a step: latency only
        dict(name="bias one layer", op="bias", L=1, S=1, E=64),
        # every layer of a deep model at once, counts kept for each sequence
        dict(name="bias all layers", op="bias", L=58, S=128, E=256),
        # the gradients of one tiny layer: latency only
        dict(name="clip tiny layer", op="clip", tensors="tiny", total=0, kind="mixed", norm=2.0),
        # hundreds of tensors of unlike sizes and types, as views of flat gradient buffers
        dict(name="clip many", op="clip", tensors="ragged", count=600, total=150_000_000, kind="mixed", norm=2.0),
        # the expert weights' gradients of a 64-expert slice of the largest layer (7168 x 2048): bf16, far beyond L2
        dict(name="clip experts", op="clip", tensors="experts", total=0, kind="bf16", norm=2.0),
        # small fp32 tensors: a router, norms and biases of a model
        dict(name="adamw small", op="adamw", tensors="ragged", count=120, total=3_000_000, kind="f32", master=False),
        # the 64-expert layer (2048 x 1408): bf16 weights and gradients, fp32 masters, clipped by the global norm
        dict(name="adamw layer", op="adamw", tensors="layer", total=0, kind="bf16", master=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route", "bias", "clip", "adamw"])
    if op == "route":
        E = rng.choice([_log(rng, 4, 1024), 8 * _log(rng, 1, 128), 32 * rng.randint(1, 32)])
        T = max(1, min(_log(rng, 1, 131072), 131072 * 128 // E))
        k = max(1, min(_log(rng, 1, 32), E))
        groups = [g for g in (2, 3, 4, 8, 16, 32) if E % g == 0 and E // g >= 2]
        n_group = rng.choice(groups) if groups and rng.random() < 0.5 else 1
        topk_group = n_group if n_group == 1 else rng.randint(max(1, -(-k * n_group // E)), n_group)
        return _route(None, T, E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(list(TYPES)),
                      normalize=rng.random() < 0.75, scale=rng.choice([1.0, 2.5]), n_group=n_group,
                      topk_group=topk_group, group_topn=rng.randint(1, min(3, E // n_group)), bias=rng.random() < 0.5,
                      S=min(T, _log(rng, 1, 64)), pad=rng.choice([0, 0, 1, 8]), masked=rng.random() < 0.4,
                      off=rng.random() < 0.3, train=rng.random() < 0.75)
    if op == "bias":
        return dict(op="bias", L=_log(rng, 1, 58), S=_log(rng, 1, 128), E=_log(rng, 2, 256))
    kind = rng.choice(["f32", "bf16", "f16", "mixed"])
    if op == "clip":
        return dict(op="clip", tensors="ragged", count=_log(rng, 1, 900), total=_log(rng, 2000, 400_000_000),
                    kind=kind, norm=rng.choice([2.0, 2.0, 1.0, float("inf")]))
    return dict(op="adamw", tensors="ragged", count=_log(rng, 1, 900), total=_log(rng, 2000, 100_000_000),
                kind=kind, master=kind != "f32" and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs


def _layout(case):
    """The sizes and types of a case's tensors, the same on every call."""
    if case["tensors"] == "tiny":        # E = 8, H = 128, I = 64
        return [(8 * 128, "f32"), (8 * 128 * 128, "bf16"), (8 * 128 * 64, "bf16")]
    if case["tensors"] == "layer":       # E = 64, H = 2048, I = 1408
        return [(64 * 2048, "bf16"), (64 * 2816 * 2048, "bf16"), (64 * 2048 * 1408, "bf16")]
    if case["tensors"] == "experts":     # 64 experts, H = 7168, I = 2048
        return [(64 * 4096 * 7168, "bf16"), (64 * 7168 * 2048, "bf16")]
    r = np.random.RandomState(case["count"] * 7919 + case["total"] % 7907)
    share = r.lognormal(0.0, 1.5, case["count"])
    sizes = np.maximum(1, (share / share.sum() * case["total"]).astype(np.int64))
    kinds = [case["kind"]] if case["kind"] != "mixed" else ["bf16", "f32", "f16"]
    return [(int(n), kinds[i % len(kinds)]) for i, n in enumerate(sizes)]


def _arenas(sizes, gen, make):
    """Tensors of the given (elements, type), as views of one flat buffer for each type."""
    arenas, views, at = {}, [], {}
    for n, t in sizes:
        at[t] = at.get(t, 0) + n
    for t in sorted(at):
        arenas[t] = make(at[t], TYPES[t], gen)
        at[t] = 0
    for n, t in sizes:
        views.append(arenas[t][at[t]:at[t] + n])
        at[t] += n
    return arenas, views


def _normal(scale):
    return lambda n, dtype, gen: torch.empty(n, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def _prepare_route(case, seed, gen):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    dtype = TYPES[case["dtype"]]
    ld = E + case["pad"]
    popular = -0.6 * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda").float()) * (case["score"] == "softmax")
    full = torch.randn((T, ld), generator=gen, device="cuda")
    full[:, :E] += popular
    if case["off"]:                      # experts that a token may not use, and tokens that may use none
        gone = torch.rand((T, E), generator=gen, device="cuda") < 0.05
        gone |= torch.rand((T, 1), generator=gen, device="cuda") < 0.01
        full[:, :E].masked_fill_(gone, -math.inf)
    r = np.random.RandomState(seed % (1 << 31))
    cuts = np.sort(r.randint(0, T + 1, S - 1)) if S > 1 else np.zeros(0, np.int64)
    offsets = torch.tensor(np.concatenate([[0], cuts, [T]]).astype(np.int32), device="cuda")
    mask = None
    if case["masked"]:                   # padding at the sequences' ends, with whatever the buffer held there
        mask = torch.rand((T,), generator=gen, device="cuda") >= 0.06
        full.masked_fill_(~mask[:, None], math.nan)
    state = dict(case=case, logits=full.to(dtype)[:, :E], mask=mask, offsets=offsets if S > 1 else None,
                 bias=0.05 * torch.randn((E,), generator=gen, device="cuda") if case["bias"] else None,
                 idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                 w=torch.empty((T, k), dtype=torch.float32, device="cuda"))
    if case["train"]:
        state.update(dw=torch.randn((T, k), generator=gen, device="cuda") / k,
                     counts=torch.empty((S, E), dtype=torch.int32, device="cuda"),
                     seq_tokens=torch.empty((S + 2,), dtype=torch.int32, device="cuda"),
                     losses=torch.empty((2,), dtype=torch.float32, device="cuda"),
                     dlosses=torch.tensor([10.0, 1.0], device="cuda") * T ** 0.5,
                     dlogits=torch.empty((T, E), dtype=dtype, device="cuda"))
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "route":
        return _prepare_route(case, seed, gen)
    if case["op"] == "bias":
        L, S, E = case["L"], case["S"], case["E"]
        return dict(case=case, bias=0.01 * torch.randn((L, E), generator=gen, device="cuda"), rate=0.001,
                    counts=torch.randint(0, 500, (L, S, E), generator=gen, device="cuda", dtype=torch.int32))
    sizes = _layout(case)
    if case["op"] == "clip":
        arenas, grads = _arenas(sizes, gen, _normal(0.01))
        scale = {1.0: 0.005 * sum(n for n, _ in sizes), 2.0: 0.006 * math.sqrt(sum(n for n, _ in sizes))}
        return dict(case=case, arenas=arenas, grads=grads, max_norm=scale.get(case["norm"], 0.03))
    pa, params = _arenas(sizes, gen, _normal(0.02))
    _, grads = _arenas(sizes, gen, _normal(0.01))
    f32 = [(n, "f32") for n, _ in sizes]
    ma, m = _arenas(f32, gen, _normal(0.001))
    va, v = _arenas(f32, gen, _normal(0.001))
    va["f32"].square_()
    state = dict(case=case, arenas=[pa, ma, va], params=params, grads=grads, m=m, v=v, masters=None,
                 step=torch.full((1,), 10, dtype=torch.int32, device="cuda"),
                 lr=torch.full((1,), 1e-3, device="cuda"), betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1,
                 max_norm=0.006 * math.sqrt(sum(n for n, _ in sizes)))
    if case["master"]:
        xa, state["masters"] = _arenas(f32, gen, lambda n, dtype, g: torch.empty(n, dtype=dtype, device="cuda"))
        state["arenas"].append(xa)
        torch._foreach_copy_(state["masters"], params)
    return state


# ---------------------------------------------------------------- plain forms


def _plain_select(state):
    """Live tokens, 32-bit scores, indices and weights."""
    c, l = state["case"], state["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    on = ~torch.isneginf(l)
    if state["mask"] is not None:
        on = on & state["mask"][:, None]
    live = on.any(1)
    # the order of near-equal experts is decided in 64 bits
    wide = torch.where(on, l, -math.inf).to(torch.float64 if state["bias"] is not None or c["n_group"] > 1 else torch.float32)
    if c["score"] == "softmax":
        top = torch.where(live[:, None], wide.amax(1, keepdim=True), 0.0)
        e = torch.exp(wide - top)
        s = e / torch.where(live[:, None], e.sum(1, keepdim=True), 1.0)
    else:
        s = 1.0 / (1.0 + torch.exp(-wide))
    sel = s + state["bias"] if state["bias"] is not None else s
    key = sel if state["bias"] is not None else wide
    key = torch.where(on, key, -math.inf)
    if c["n_group"] > 1:
        size = E // c["n_group"]
        best = torch.where(on, sel, -math.inf).view(T, c["n_group"], size).sort(dim=2, descending=True)[0][:, :, :c["group_topn"]]
        total = torch.where(torch.isneginf(best), 0.0, best).sum(2)
        total = torch.where(torch.isneginf(best[:, :, 0]), -math.inf, total)
        kept = total.sort(dim=1, descending=True, stable=True)[1][:, :c["topk_group"]]
        allowed = torch.zeros((T, c["n_group"]), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(allowed.repeat_interleave(size, 1), key, -math.inf)
    value, order = key.sort(dim=1, descending=True, stable=True)
    idx = torch.where(torch.isneginf(value[:, :k]), -1, order[:, :k]).int()
    s = s.float()
    chosen = torch.where(idx >= 0, s.gather(1, order[:, :k]), 0.0)
    w = chosen * c["scale"]
    if c["normalize"]:
        w = chosen / (chosen.sum(1, keepdim=True) + 1e-20) * c["scale"]
    return on, live, s, idx, w


def _plain_route(state):
    c, l = state["case"], state["logits"]
    T, E, k, S, scale = c["T"], c["E"], c["k"], c["S"], c["scale"]
    on, live, s, idx, w = _plain_select(state)
    if not c["train"]:
        return [idx, w]
    if state["offsets"] is not None:
        seq = torch.searchsorted(state["offsets"][1:-1], torch.arange(T, dtype=torch.int32, device=l.device), right=True)
    else:
        seq = torch.zeros((T,), dtype=torch.int64, device=l.device)
    n = torch.zeros((S,), dtype=torch.int64, device=l.device).index_add_(0, seq, live.long())
    flat = torch.where(idx >= 0, seq[:, None] * E + idx, S * E).flatten()
    counts = torch.bincount(flat, minlength=S * E + 1)[:S * E].view(S, E)
    N, used = n.sum(), (n > 0).sum()
    # balance and z; long sums in 64 bits
    nf = n.clamp(min=1).double()
    Z = torch.where(live, s.sum(1), 1.0)[:, None]
    share = s / Z
    P = torch.zeros((S, E), dtype=torch.float64, device=l.device).index_add_(0, seq, share.double()) / nf[:, None]
    f = E * counts.double() / (k * nf[:, None])
    l32 = torch.where(on, l, -math.inf).float()
    top = torch.where(live[:, None], l32.amax(1, keepdim=True), 0.0)
    ex = torch.exp(l32 - top)
    exsum = torch.where(live, ex.sum(1), 1.0)[:, None]
    lse = torch.where(live[:, None], top + torch.log(exsum), 0.0)
    losses = torch.stack([(f * P).sum() / used.clamp(min=1), lse.double().square().sum() / N.clamp(min=1)]).float()
    # the backward, for the weights' gradient and the two terms'
    dbal, dz = state["dlosses"]
    at = idx.clamp(min=0).long()
    chosen = torch.where(idx >= 0, s.gather(1, at), 0.0)
    dw = torch.where(idx >= 0, state["dw"], 0.0)
    if c["normalize"]:
        total = chosen.sum(1, keepdim=True) + 1e-20
        gw = scale / total * (dw - (dw * chosen / total).sum(1, keepdim=True))
    else:
        gw = scale * dw
    gs = torch.zeros((T, E), device=l.device).scatter_add_(1, at, torch.where(idx >= 0, gw, 0.0))
    a = (dbal * (f / nf[:, None] / used.clamp(min=1))).float()[seq]
    if c["score"] == "softmax":
        gs = gs + a
        dl = s * (gs - (s * gs).sum(1, keepdim=True))
    else:
        gs = gs + (a - (share * a).sum(1, keepdim=True)) / Z
        dl = s * (1.0 - s) * gs
    dl = dl + dz * 2.0 / N.clamp(min=1) * lse * (ex / exsum)
    dl = torch.where(on, dl, 0.0)
    return [idx, w, counts.int(), torch.cat([n, N[None], used[None]]).int(), losses, dl.to(l.dtype)]


def _plain_bias(state):
    c = state["counts"].sum(1)
    E = state["case"]["E"]
    state["bias"].add_(torch.sign(c.sum(1, keepdim=True) - E * c).float() * state["rate"])
    return state["bias"]


def _plain_norm(grads, p):
    if p == 2.0:
        return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()
    if p == 1.0:
        return torch.stack([g.float().abs().sum(dtype=torch.float64) for g in grads]).sum().float()
    return torch.stack([g.float().abs().max() for g in grads]).max()


def _outputs(state):
    return [a[t] for a in (state["arenas"] if isinstance(state["arenas"], list) else [state["arenas"]]) for t in sorted(a)]


def _plain_clip(state):
    norm = _plain_norm(state["grads"], state["case"]["norm"])
    f = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
    [g.copy_(g.float() * f) for g in state["grads"]]
    return _outputs(state) + [norm]


def _plain_adamw_one(state, p, g, m, v, x, f, c1, c2):
    b1, b2 = state["betas"]
    g = g.float() * f
    m.copy_(b1 * m + (1.0 - b1) * g)
    v.copy_(b2 * v + (1.0 - b2) * g * g)
    old = x if x is not None else p.float()
    new = old - state["lr"] * (state["weight_decay"] * old + (m / c1) / (torch.sqrt(v / c2) + state["eps"]))
    if x is not None:
        x.copy_(new)
    p.copy_(new)


def _plain_adamw(state):
    norm = _plain_norm(state["grads"], 2.0)
    f = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
    state["step"].add_(1)
    c1, c2 = ((1.0 - torch.pow(torch.tensor(b, dtype=torch.float64, device="cuda"), state["step"])).float() for b in state["betas"])
    xs = state["masters"] or [None] * len(state["params"])
    [_plain_adamw_one(state, *t, f, c1, c2) for t in zip(state["params"], state["grads"], state["m"], state["v"], xs)]
    return _outputs(state) + [norm]


# ---------------------------------------------------------------- the framework's calls


def _own_route(state):
    from moe_expert_router_gb300 import binding as B
    c = state["case"]
    cfg = B.router_cfg(c["score"], c["normalize"], c["scale"], c["n_group"], c["topk_group"], c["group_topn"])
    if not c["train"]:
        B.moe_route(state["logits"], cfg, state["idx"], state["w"], sel_bias=state["bias"], token_mask=state["mask"])
        return [state["idx"], state["w"]]
    if "ws" not in state:
        state["ws"] = torch.empty(B.moe_route_workspace_size(c["T"], c["E"], c["S"]), dtype=torch.uint8, device="cuda")
    B.moe_route(state["logits"], cfg, state["idx"], state["w"], sel_bias=state["bias"], token_mask=state["mask"],
                seq_offsets=state["offsets"], counts=state["counts"], seq_tokens=state["seq_tokens"],
                losses=state["losses"], ws=state["ws"])
    B.moe_route_backward(state["logits"], cfg, state["idx"], state["dw"], state["dlogits"], token_mask=state["mask"],
                         seq_offsets=state["offsets"], counts=state["counts"], seq_tokens=state["seq_tokens"],
                         dlosses=state["dlosses"])
    return [state[n] for n in ("idx", "w", "counts", "seq_tokens", "losses", "dlogits")]


def _own_bias(state):
    from moe_expert_router_gb300 import binding as B
    B.moe_bias_update(state["bias"], state["counts"], state["rate"])
    return state["bias"]


def _own_clip(state):
    from moe_expert_router_gb300 import optim
    return _outputs(state) + [optim.clip_grad_norm_(state["grads"], state["max_norm"], state["case"]["norm"])]


def _own_adamw(state):
    from moe_expert_router_gb300 import optim
    norm = optim.adamw_step(state["params"], state["grads"], state["m"], state["v"], state["step"], state["lr"],
                            masters=state["masters"], betas=state["betas"], eps=state["eps"],
                            weight_decay=state["weight_decay"], max_norm=state["max_norm"])
    return _outputs(state) + [norm]


def run(state):
    op = state["case"]["op"]
    if op == "clip":
        # gradients that a pass has clipped come back: the next bound is lower, so that every pass clips
        state["max_norm"] *= 0.99
    if own:
        return {"route": _own_route, "bias": _own_bias, "clip": _own_clip, "adamw": _own_adamw}[op](state)
    return {"route": _plain_route, "bias": _plain_bias, "clip": _plain_clip, "adamw": _plain_adamw}[op](state)


def work(case):
    if case["op"] == "route":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        size = TYPES[case["dtype"]].itemsize
        read = T * E * size + T * case["masked"] + 4 * E * case["bias"]
        if not case["train"]:
            return {"bytes": read + 8 * T * k, "flops": 10.0 * T * E}
        return {"bytes": read + 12 * T * k + 4 * S * E + T * E * size, "flops": 40.0 * T * E}
    if case["op"] == "bias":
        return {"bytes": 4 * case["L"] * (case["S"] + 2) * case["E"], "flops": case["L"] * case["S"] * case["E"]}
    sizes = _layout(case)
    if case["op"] == "clip":
        return {"bytes": sum(2 * n * TYPES[t].itemsize for n, t in sizes), "flops": 3.0 * sum(n for n, _ in sizes)}
    each = {t: 3 * TYPES[t].itemsize + 16 if not case["master"] else 2 * TYPES[t].itemsize + 24 for t in TYPES}
    return {"bytes": sum(n * each[t] for n, t in sizes), "flops": 20.0 * sum(n for n, _ in sizes)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _exact_route(state):
    c = state["case"]
    T, E, k, S, scale = c["T"], c["E"], c["k"], c["S"], c["scale"]
    l = _np(state["logits"])
    alive = np.ones(T, bool) if state["mask"] is None else state["mask"].cpu().numpy()
    l = np.where(alive[:, None], l, -np.inf)
    on = l > -np.inf
    alive = on.any(1)
    peak = np.where(alive, l.max(1), 0.0)[:, None]
    ex = np.where(on, np.exp(np.where(on, l, 0.0) - peak), 0.0)
    soft = ex / np.where(alive, ex.sum(1), 1.0)[:, None]
    s = soft if c["score"] == "softmax" else np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l, 0.0))), 0.0)
    shifted = s + (0.0 if state["bias"] is None else _np(state["bias"]))
    rank = np.where(on, l if state["bias"] is None else shifted, -np.inf)
    if c["n_group"] > 1:
        size = E // c["n_group"]
        inside = -np.sort(-np.where(on, shifted, -np.inf).reshape(T, c["n_group"], size), axis=2)[:, :, :c["group_topn"]]
        sums = np.where(np.isinf(inside[:, :, 0]), -np.inf, np.where(np.isinf(inside), 0.0, inside).sum(2))
        lost = np.argsort(-sums, axis=1, kind="stable")[:, c["topk_group"]:]
        stays = np.ones((T, c["n_group"]), bool)
        np.put_along_axis(stays, lost, False, 1)
        rank = np.where(np.repeat(stays, size, 1), rank, -np.inf)
    pick = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    filled = np.take_along_axis(rank, pick, 1) > -np.inf
    sk = np.where(filled, np.take_along_axis(s, pick, 1), 0.0)
    base = sk.sum(1, keepdims=True) + 1e-20 if c["normalize"] else np.ones((T, 1))
    w = scale * sk / base
    if not c["train"]:
        return [None, w]
    edges = np.array([0, T]) if state["offsets"] is None else state["offsets"].cpu().numpy()
    length = np.diff(edges)
    owner = np.repeat(np.arange(S), length)
    n = np.array([alive[edges[b]:edges[b + 1]].sum() for b in range(S)])
    share = s / np.where(alive, s.sum(1), 1.0)[:, None]
    hits = np.zeros((T, E))
    np.put_along_axis(hits, pick, filled.astype(float), 1)
    hits = np.stack([hits[edges[b]:edges[b + 1]].sum(0) for b in range(S)])
    P = np.stack([share[edges[b]:edges[b + 1]].sum(0) for b in range(S)])
    N, used, nn = max(1, n.sum()), max(1, (n > 0).sum()), np.maximum(n, 1)[:, None].astype(float)
    lse = np.where(alive, peak[:, 0] + np.log(np.where(alive, ex.sum(1), 1.0)), 0.0)
    losses = np.array([(E * hits * P / (k * nn * nn)).sum() / used, (lse ** 2).sum() / N])
    dbal, dz = _np(state["dlosses"])
    dw = np.where(filled, _np(state["dw"]), 0.0)
    gk = scale / base * (dw - (dw * sk).sum(1, keepdims=True) / base * c["normalize"])
    g = np.zeros((T, E))
    np.put_along_axis(g, pick, np.where(filled, gk, 0.0), 1)
    ga = (dbal * E * hits / (k * nn * nn * used))[owner]
    gs = g + (ga - (share * ga).sum(1, keepdims=True)) / np.where(alive, s.sum(1), 1.0)[:, None]
    dl = s * (gs - (s * gs).sum(1, keepdims=True)) if c["score"] == "softmax" else s * (1.0 - s) * gs
    dl = np.where(on, dl + dz * 2.0 / N * lse[:, None] * soft, 0.0)
    return [None, w, None, None, losses, dl]


def _exact_norm(grads, p):
    if p == 2.0:
        return np.sqrt(sum(float(np.dot(g, g)) for g in grads))
    return sum(float(np.abs(g).sum()) for g in grads) if p == 1.0 else max(float(np.abs(g).max()) for g in grads)


def exact(case, seed):
    if case["op"] in ("clip", "adamw") and sum(n for n, _ in _layout(case)) > 200_000_000:
        return None
    state = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(state)
    if case["op"] == "bias":
        c = state["counts"].cpu().numpy().astype(np.int64).sum(1)
        return _np(state["bias"]) + state["rate"] * np.sign(c.sum(1, keepdims=True) - case["E"] * c)
    if case["op"] == "clip":
        flat = {t: _np(a) for t, a in state["arenas"].items()}
        norm = _exact_norm(list(flat.values()), case["norm"])
        f = min(1.0, state["max_norm"] * 0.99 / (norm + 1e-6))
        return [flat[t] * f for t in sorted(flat)] + [np.array(norm)]
    grads = [_np(g) for g in state["grads"]]
    norm = _exact_norm(grads, 2.0)
    f = min(1.0, state["max_norm"] / (norm + 1e-6))
    (b1, b2), t = state["betas"], int(state["step"]) + 1
    pa, ma, va = state["arenas"][:3]
    out_p, out_m, out_v = {k: _np(a) for k, a in pa.items()}, _np(ma["f32"]), _np(va["f32"])
    at, by = 0, {k: 0 for k in out_p}
    lr, masters = float(state["lr"]), np.zeros(out_m.size) if case["master"] else None
    for (n, kind), g in zip(_layout(case), grads):
        g = g * f
        sl, ps = slice(at, at + n), slice(by[kind], by[kind] + n)
        out_m[sl] = b1 * out_m[sl] + (1 - b1) * g
        out_v[sl] = b2 * out_v[sl] + (1 - b2) * g * g
        p = out_p[kind][ps]
        p = p - lr * (state["weight_decay"] * p + out_m[sl] / (1 - b1 ** t) / (np.sqrt(out_v[sl] / (1 - b2 ** t)) + state["eps"]))
        out_p[kind][ps] = p
        if masters is not None:
            masters[sl] = p
        at, by[kind] = at + n, by[kind] + n
    return [out_p[k] for k in sorted(out_p)] + [out_m, out_v] + ([masters] if masters is not None else []) + [np.array(norm)]
