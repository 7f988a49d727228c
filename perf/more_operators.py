"""Cases of the norm in front of the expert layer and of products grouped by expert.

Three operators: the root-mean-square norm of a residual stream (`norm`: the addition of
a branch's output, the norm, and where asked for the MXFP8 form of the result that the
MXFP8 products read; forward alone as serving calls it, or forward and backward), the
products of rows with the matrix of their group (`grouped`: forward alone, or with the
gradients of rows and matrices), and the same products of MXFP8 operands (`grouped_mx`).

`run` computes them in elementary torch operations, or, where `own` is true, through this
repository's package.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def _norm(name, T, H, dtype, **more):
    case = dict(op="norm", T=T, H=H, dtype=dtype, weight="f32", residual=True, mx=False, train=False, pad=0)
    case.update(more)
    return {"name": name, **case} if name else case


def _grouped(name, R, G, K, N, dtype, **more):
    case = dict(op="grouped", R=R, G=G, K=K, N=N, dtype=dtype, layout="nk", train=False, skew=0.5, pad=0, tail=0)
    case.update(more)
    return {"name": name, **case} if name else case


def listed():
    return [
        # one token in front of the widest expert layer while it generates: latency only
        _norm("norm one token", 1, 7168, "bf16"),
        # a batch of 64 generating requests, the result also in MXFP8 for the experts
        _norm("norm decode mx", 64, 4096, "bf16", mx=True),
        # a prompt's 8192 tokens at the widest layer, the result also in MXFP8
        _norm("norm prompt mx", 8192, 7168, "bf16", mx=True),
        # a training step of the 2048-wide model, forward and backward
        _norm("norm train", 4096, 2048, "bf16", train=True),
        # odd sizes: a width that no vector divides, rows wider than it, fp16, no branch to add
        _norm("norm train odd", 5003, 1003, "f16", weight="f16", residual=False, train=True, pad=6),
        # the longest batch of a training step, forward and backward
        _norm("norm train long", 32768, 4096, "bf16", weight="bf16", train=True),
        # one generated token through its 8 of 32 experts at the widest layer: the matrices' bytes
        _grouped("grouped one token", 8, 32, 7168, 4096, "bf16", skew=0.0),
        # 64 generating requests, 8 experts each of 128, some popular
        _grouped("grouped decode", 512, 128, 4096, 1536, "bf16", skew=1.2),
        # small ragged groups of a fp16 model, matrices stored input by output, rows left over
        _grouped("grouped ragged", 5003, 11, 264, 520, "f16", layout="kn", train=True, skew=1.0, pad=8, tail=37),
        # a training step's products of the 64-expert layer, forward and both gradients
        _grouped("grouped train", 24576, 64, 2048, 2816, "bf16", train=True),
        # a few requests of the 64-expert model in MXFP8
        dict(name="grouped mx batch", op="grouped_mx", R=1000, G=64, K=2048, N=1408, skew=1.0),
        # a prompt's rows at the widest layer in MXFP8, 32 experts
        dict(name="grouped mx prompt", op="grouped_mx", R=8192, G=32, K=7168, N=4096, skew=0.5),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "grouped", "grouped", "grouped_mx"])
    if op == "norm":
        mx = rng.random() < 0.3
        H = 128 * _log(rng, 1, 64) if mx else rng.choice([_log(rng, 8, 8192), 8 * _log(rng, 1, 1024)])
        T = max(1, min(_log(rng, 1, 32768), 32768 * 4096 // (2 * H)))
        dtype = rng.choice(list(TYPES))
        return _norm(None, T, H, dtype, weight=rng.choice(["f32", dtype]), residual=rng.random() < 0.7, mx=mx,
                     train=not mx and rng.random() < 0.6, pad=rng.choice([0, 0, 0, 8, 5]))
    if op == "grouped":
        G, K, N = _log(rng, 1, 128), 8 * _log(rng, 2, 896), 8 * _log(rng, 2, 512)
        G = max(1, min(G, 128 * 4096 * 1536 // (K * N)))
        train = rng.random() < 0.5
        R = max(1, min(_log(rng, 1, 24576), 24576 * 2048 * 2816 // (K * N)))
        return _grouped(None, R, G, K, N, rng.choice(["bf16", "bf16", "f16"]), layout=rng.choice(["nk", "nk", "kn"]),
                        train=train, skew=rng.choice([0.0, 0.5, 1.0]), pad=rng.choice([0, 0, 8, 24]),
                        tail=rng.choice([0, 0, 1, 50]) if R > 100 else 0)
    G, K, N = _log(rng, 1, 64), 128 * _log(rng, 1, 56), 8 * _log(rng, 2, 512)
    G = max(1, min(G, 64 * 2048 * 4096 // (K * N)))
    R = max(1, min(_log(rng, 1, 8192), 8192 * 7168 * 4096 // (K * N)))
    return dict(op="grouped_mx", R=R, G=G, K=K, N=N, skew=rng.choice([0.0, 0.5, 1.0]))


# ---------------------------------------------------------------- MXFP8


def _mx(v):
    """OCP MXFP8 of v [..., cols] along its last dimension, cols a multiple of 32: E4M3 values
    and the E8M0 codes [..., cols / 32] of 2^(floor(log2 max|v|) - 8)."""
    b = v.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = (torch.frexp(top)[1] - 9).clamp(-127, 127)                     # frexp: top = m 2^e, m in [1/2, 1)
    e = torch.where(top == 0, -127, e)
    scaled = torch.ldexp(b.double(), -e[..., None].double()).clamp(-448.0, 448.0).float()
    return scaled.to(torch.float8_e4m3fn).flatten(-2), (e + 127).to(torch.uint8)


def _words(sc):
    """E8M0 codes [rows, cols / 32] in the order that the products read: [cols / 128, rows up to 4s, 4]."""
    rows, blocks = sc.shape
    out = torch.zeros((blocks // 4, -(-rows // 4) * 4, 4), dtype=torch.uint8, device=sc.device)
    out[:, :rows] = sc.view(rows, blocks // 4, 4).permute(1, 0, 2)
    return out


def _values(codes, words):
    """The fp32 values of E4M3 codes [rows, cols] with their scale words."""
    rows, cols = codes.shape
    e = words.view(cols // 128, -1, 4)[:, :rows].permute(1, 0, 2).reshape(rows, cols // 32)
    two = torch.pow(2.0, e.double() - 127.0)
    return (codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 32)) * two.float()[..., None]).flatten(1)


# ---------------------------------------------------------------- inputs


def _randn(gen, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)


def _wide(gen, rows, cols, dtype, pad, scale=1.0):
    """Rows of `cols` values that lie cols + pad apart."""
    return _randn(gen, (rows, cols + pad), dtype, scale)[:, :cols]


def _sizes(case):
    """Rows of each group in falling order, the same on every call: a Zipf law of the given skew."""
    rows, G = case["R"] - case.get("tail", 0), case["G"]
    share = (1.0 + np.arange(G)) ** -case["skew"]
    n = np.floor(share / share.sum() * rows).astype(np.int64)
    n[:rows - int(n.sum())] += 1
    return n


def _offsets(case, seed):
    n = np.random.RandomState(seed % (1 << 31)).permutation(_sizes(case))
    offsets = np.concatenate([[0], np.cumsum(n)])
    group = np.repeat(np.arange(case["G"]), n)
    place = np.arange(len(group)) - offsets[group]
    cuda = lambda a, t: torch.tensor(a.astype(t), device="cuda")  # noqa: E731
    # the widest group and each row's place in it serve the plain form, which pads the groups
    return {"offsets": cuda(offsets, np.int32), "group": cuda(group, np.int64), "place": cuda(place, np.int64),
            "most": int(n.max()), "rows": len(group)}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm":
        T, H, dtype = case["T"], case["H"], TYPES[case["dtype"]]
        # a residual stream: some columns are far larger than the others
        wide = torch.exp(0.8 * _randn(gen, (H,), torch.float32))
        state["x"] = _wide(gen, T, H, dtype, case["pad"])
        state["x"].mul_(wide.to(dtype))
        state["residual"] = _wide(gen, T, H, dtype, case["pad"]) if case["residual"] else None
        state["weight"] = (1.0 + _randn(gen, (H,), torch.float32, 0.3)).to(TYPES[case["weight"]])
        buffer = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        state["y"] = buffer((T, H), dtype)
        state["h"] = buffer((T, H), dtype) if case["residual"] else None
        state["rstd"] = buffer((T,), torch.float32) if case["train"] else None
        if case["mx"]:
            state["codes"] = buffer((T, H), torch.uint8)
            state["scales"] = buffer((H // 128, -(-T // 4) * 4, 4), torch.uint8)
        if case["train"]:
            state["dy"] = _randn(gen, (T, H), dtype)
            state["dh"] = _randn(gen, (T, H), dtype) if case["residual"] else None
            state["dx"], state["dweight"] = buffer((T, H), dtype), buffer((H,), TYPES[case["weight"]])
        return state
    state.update(_offsets(case, seed))
    R, G, K, N = case["R"], case["G"], case["K"], case["N"]
    if case["op"] == "grouped_mx":
        codes, sc = _mx(_randn(gen, (R, K), torch.bfloat16))
        state["x"], state["x_scales"] = codes.view(torch.uint8), _words(sc)
        state["w"] = torch.empty((G * N, K), dtype=torch.uint8, device="cuda")
        sc = torch.empty((G * N, K // 32), dtype=torch.uint8, device="cuda")
        for r in range(0, G * N, 8192):
            some = _mx(_randn(gen, (min(8192, G * N - r), K), torch.bfloat16, K ** -0.5))
            state["w"][r:r + 8192], sc[r:r + 8192] = some[0].view(torch.uint8), some[1]
        state["w_scales"] = _words(sc)
        state["out"] = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    else:
        dtype, pad = TYPES[case["dtype"]], case["pad"]
        state["x"] = _wide(gen, R, K, dtype, pad)
        state["w"] = _randn(gen, (G, N, K) if case["layout"] == "nk" else (G, K, N), dtype, K ** -0.5)
        state["out"] = torch.zeros((R, N), dtype=dtype, device="cuda")
        if case["train"]:
            state["dy"] = _wide(gen, R, N, dtype, pad)
            state["dx"] = torch.zeros((R, K), dtype=dtype, device="cuda")
            state["dw"] = torch.zeros_like(state["w"])
    state["ws"] = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")   # enough for any number of groups
    return state


# ---------------------------------------------------------------- the plain forms


def _rounded(v, dtype):
    """64-bit values rounded once to a type that a conversion would reach through fp32."""
    f = v.float()
    if dtype == torch.float32:
        return f
    low = v - f.double()
    bits = f.view(torch.int32)
    odd = torch.where((bits & 1 == 0) & (low != 0), torch.sign(low * f.double()).int(), 0)
    return (bits + odd).view(torch.float32).to(dtype)


def _plain_norm(state):
    c, x = state["case"], state["x"]
    dtype = x.dtype
    h = x if state["residual"] is None else (x.float() + state["residual"].float()).to(dtype)
    # in 64 bits: y lies next to a border between two values of its type now and then
    rstd = 1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)
    y = _rounded(h.double() * rstd * state["weight"].double(), dtype)
    out = {"y": y}
    if state["residual"] is not None:
        out["h"] = h
    if c["mx"]:
        codes, sc = _mx(y)
        out["codes"], out["scales"] = codes, _words(sc)[:, :c["T"]].view(torch.float8_e8m0fnu)
    if c["train"]:
        r, h32, dy = rstd.float(), h.float(), state["dy"].float()
        g = dy * state["weight"].float()
        dx = r * (g - h32 * (r * r * (g * h32).mean(1, keepdim=True)))
        if state["dh"] is not None:
            dx = dx + state["dh"].float()
        out["dx"] = dx.to(dtype)
        out["dweight"] = (dy * h32 * r).sum(0, dtype=torch.float64).to(state["weight"].dtype)
    return out


def _padded(state, rows):
    """Rows [R, cols] as [G, widest, cols], zeros behind each group's own."""
    c = state["case"]
    out = torch.zeros((c["G"], state["most"], rows.shape[1]), dtype=torch.float32, device=rows.device)
    out[state["group"], state["place"]] = rows[:state["rows"]].float()
    return out


def _unpadded(state, v, into):
    into[:state["rows"]] = v[state["group"], state["place"]].to(into.dtype)
    return into


def _plain_grouped(state):
    c = state["case"]
    w = state["w"].float() if c["layout"] == "kn" else state["w"].float().transpose(1, 2)
    x = _padded(state, state["x"])
    out = {"out": _unpadded(state, torch.bmm(x, w), state["out"])}
    if c["train"]:
        dy = _padded(state, state["dy"])
        out["dx"] = _unpadded(state, torch.bmm(dy, w.transpose(1, 2)), state["dx"])
        a, b = (x, dy) if c["layout"] == "kn" else (dy, x)
        out["dw"] = torch.bmm(a.transpose(1, 2), b).to(state["dw"].dtype)
    return out


def _plain_grouped_mx(state):
    c = state["case"]
    w = _values(state["w"], state["w_scales"]).view(c["G"], c["N"], c["K"])
    x = _padded(state, _values(state["x"], state["x_scales"]))
    return {"out": _unpadded(state, torch.bmm(x, w.transpose(1, 2)), state["out"])}


# ---------------------------------------------------------------- the framework's calls


def _own_norm(state):
    from moe_expert_router_gb300 import binding as B
    c = state["case"]
    s = state
    out = {"y": s["y"]}
    if c["mx"]:
        B.moe_rms_norm(s["x"], s["weight"], s["y"], EPS, residual=s["residual"], h=s["h"], codes=s["codes"],
                       scales=s["scales"])
        out["codes"] = s["codes"].view(torch.float8_e4m3fn)
        out["scales"] = s["scales"][:, :c["T"]].view(torch.float8_e8m0fnu)
    else:
        B.moe_rms_norm(s["x"], s["weight"], s["y"], EPS, residual=s["residual"], h=s["h"], rstd=s["rstd"])
    if s["h"] is not None:
        out["h"] = s["h"]
    if c["train"]:
        h = s["x"] if s["h"] is None else s["h"]
        B.moe_rms_norm_backward(s["dy"], h, s["weight"], s["rstd"], s["dx"], s["dweight"],
                                B.rms_norm_scratch(c["T"], c["H"], s["dx"]), dh=s["dh"])
        out["dx"], out["dweight"] = s["dx"], s["dweight"]
    return out


def _own_grouped(state):
    from moe_expert_router_gb300 import binding as B
    s, kn = state, state["case"]["layout"] == "kn"
    B.moe_grouped_mm(s["x"], s["w"], s["offsets"], s["out"], s["ws"], transposed=kn)
    out = {"out": s["out"]}
    if s["case"]["train"]:
        B.moe_grouped_mm(s["dy"], s["w"], s["offsets"], s["dx"], s["ws"], transposed=not kn)
        a, b = (s["x"], s["dy"]) if kn else (s["dy"], s["x"])
        B.moe_grouped_wgrad(a, b, s["offsets"], s["dw"], s["ws"])
        out["dx"], out["dw"] = s["dx"], s["dw"]
    return out


def _own_grouped_mx(state):
    from moe_expert_router_gb300 import binding as B
    s, c = state, state["case"]
    B.moe_grouped_mm_mx(s["x"], s["x_scales"], s["w"].view(c["G"], c["N"], c["K"]), s["w_scales"], s["offsets"],
                        s["out"], s["ws"])
    return {"out": s["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "grouped": _own_grouped, "grouped_mx": _own_grouped_mx}[op](state)
    return {"norm": _plain_norm, "grouped": _plain_grouped, "grouped_mx": _plain_grouped_mx}[op](state)


# ---------------------------------------------------------------- in 64 bits


def _floor_log2(v):
    """Of positive normal 64-bit values, from their bits: log2 itself may fall short of a whole number."""
    return ((v.view(torch.int64) >> 52) - 1023).double()


def _e4m3_64(v):
    """E4M3 values (in 64 bits) and 2^e of MXFP8, from the format: steps of 2^(floor(log2) - 3), no finer than 2^-9."""
    b = v.view(v.shape[0], -1, 32)
    top = b.abs().max(2).values
    e = torch.where(top > 0, _floor_log2(torch.where(top > 0, top, 1.0)) - 8.0, -127.0).clamp(-127.0, 127.0)
    s = (b / torch.exp2(e)[:, :, None]).clamp(-448.0, 448.0)
    step = torch.exp2(_floor_log2(s.abs().clamp(min=2.0 ** -6)) - 3.0)
    return (torch.round(s / step) * step).view_as(v), torch.exp2(e)


def _exact_norm(state):
    c = state["case"]
    x, w, T, H = state["x"].double(), state["weight"].double(), c["T"], c["H"]
    out, h = {}, x
    if state["residual"] is not None:
        out["h"] = x + state["residual"].double()
        h = (state["x"].float() + state["residual"].float()).to(state["x"].dtype).double()   # the stream as it is kept
    n = torch.rsqrt((h * h).sum(1) / H + EPS)[:, None]
    out["y"] = h * n * w
    if c["mx"]:
        codes, two = _e4m3_64(_rounded(out["y"], state["x"].dtype).double())
        out["codes"] = codes
        out["scales"] = two.view(T, H // 128, 4).transpose(0, 1).contiguous()
    if c["train"]:
        dy = state["dy"].double()
        z = h * n                                                      # the normalised stream
        out["dweight"] = (dy * z).sum(0)
        dz = dy * w
        out["dx"] = (dz - z * (dz * z).sum(1, keepdim=True) / H) * n
        if state["dh"] is not None:
            out["dx"] += state["dh"].double()
    return out


def _exact_grouped(state):
    c = state["case"]
    offsets = state["offsets"].tolist()
    mx = c["op"] == "grouped_mx"
    R, G, K, N = c["R"], c["G"], c["K"], c["N"]
    out = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    dx, dw = None, None
    if not mx and c["train"]:
        dx = torch.zeros((R, K), dtype=torch.float64, device="cuda")
        dw = torch.zeros(state["w"].shape, dtype=torch.float64, device="cuda")
    x = _values(state["x"], state["x_scales"]) if mx else state["x"]
    w_mx = _values(state["w"], state["w_scales"]).view(G, N, K) if mx else None
    for g in range(G):
        a, b = offsets[g], offsets[g + 1]
        if a == b:
            continue
        w = (w_mx if mx else state["w"])[g].double()
        w = w if not mx and c["layout"] == "kn" else w.t()
        out[a:b] = x[a:b].double() @ w
        if dx is not None:
            dy = state["dy"][a:b].double()
            dx[a:b] = dy @ w.t()
            d = x[a:b].double().t() @ dy
            dw[g] = d if c["layout"] == "kn" else d.t()
    return {"out": out} if dx is None else {"out": out, "dx": dx, "dw": dw}


def exact(case, seed):
    if case["op"] != "norm" and 2.0 * case["R"] * case["K"] * case["N"] > 1e12:
        return None
    state = prepare(case, seed)
    return _exact_norm(state) if case["op"] == "norm" else _exact_grouped(state)


def work(case):
    if case["op"] == "norm":
        T, H, b = case["T"], case["H"], 4 if case["dtype"] == "f32" else 2
        wide = T * H * b
        more = case["residual"]
        total = wide * (2 + 2 * more)                                  # x, y; the branch and the new stream
        flops = 4 * T * H
        if case["mx"]:
            total += T * H + T * H // 32
        if case["train"]:
            total += wide * (2 + more)                                 # dy, dx; the stream's own gradient
            flops += 9 * T * H
        return {"bytes": total + (1 + case["train"]) * H * (4 if case["weight"] == "f32" else 2), "flops": flops}
    R, K, N = case["R"] - case.get("tail", 0), case["K"], case["N"]
    used = int((_sizes(case) > 0).sum())
    if case["op"] == "grouped_mx":
        return {"bytes": (R * K + used * N * K) * 33 / 32 + 2 * R * N, "flops": 2 * R * K * N}
    if case["train"]:
        return {"bytes": 2 * (2 * R * K + 2 * R * N + (used + case["G"]) * K * N), "flops": 6 * R * K * N}
    return {"bytes": 2 * (R * K + used * K * N + R * N), "flops": 2 * R * K * N}
