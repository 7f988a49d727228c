"""The trainable router and the list operators on a host without a GPU: their formulas
against differences, their shape functions, and every refusal (arguments are checked before
the device is touched)."""
import ctypes

import numpy as np
import pytest
import torch

import route_reference as R
from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import build as moe_build
from moe_expert_router_gb300 import optim, torch_ops


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.load()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_reference_gradient_is_that_of_differences(score, normalize):
    rng = np.random.default_rng(3)
    T, E, k = 9, 7, 3
    l = rng.normal(size=(T, E))
    l[2, 4] = -np.inf
    l[5, :] = -np.inf
    mask = np.ones(T, bool)
    mask[7] = False
    off = [0, 4, 4, 9]
    dw = rng.normal(size=(T, k))
    r = R.route(l, k, score, normalize, 1.7, mask=mask, offsets=off)
    grad, _ = R.route_backward(l, r, dw, 3.0, 0.7, k, score, normalize, 1.7, off)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert grad[t, e] == 0.0
                continue
            hi, lo = l.copy(), l.copy()
            hi[t, e] += h
            lo[t, e] -= h
            d = (R.chosen_value(hi, r, dw, 3.0, 0.7, k, score, normalize, 1.7, off)
                 - R.chosen_value(lo, r, dw, 3.0, 0.7, k, score, normalize, 1.7, off)) / (2 * h)
            # truncation h^2 and the differences' rounding, value * 2^-53 / h
            assert abs(d - grad[t, e]) < 1e-8


def test_reference_balance_limits():
    # every share equal and every expert chosen equally often: 1; one expert takes all: E / k
    r = R.route(np.zeros((4, 4)), 4)
    assert abs(r["losses"][0] - 1.0) < 1e-12 and abs(r["losses"][1] - np.log(4.0) ** 2) < 1e-12
    l = np.full((6, 5), -50.0)
    l[:, 2] = 50.0
    assert abs(R.route(l, 1)["losses"][0] - 5.0) < 1e-12


P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
PAIR = ctypes.c_void_p((1 << 20) + 2)


def _route_call(lib, shape, cfg=None, logits=P, idx=P, w=P, counts=None, tokens=None, losses=None, ws=None, n=0,
                off=None, bias=None):
    cfg = B.router_cfg() if cfg is None else cfg
    return lib.moe_route(logits, bias, None, off, ctypes.byref(shape), ctypes.byref(cfg), idx, w, counts, tokens, losses,
                         ws, n, None)


def _shape(T=16, E=8, S=1, ld=8, k=2, dtype=0):
    return B.RouteShape(T, E, S, ld, k, dtype)


@pytest.mark.parametrize("shape,status", [
    (_shape(T=-1), 1), (_shape(E=0, k=1), 1), (_shape(S=0), 1), (_shape(ld=7), 1), (_shape(k=0), 1), (_shape(dtype=3), 1),
    (_shape(dtype=-1), 1), (_shape(E=1025, ld=1025), 2), (_shape(k=9), 2), (_shape(E=64, ld=64, k=33), 2),
    (_shape(T=(1 << 30) + 1), 2), (_shape(S=(1 << 24) + 1), 2),
])
def test_route_refuses_shapes(lib, shape, status):
    n = ctypes.c_size_t()
    assert lib.moe_route_workspace_size(ctypes.byref(shape), ctypes.byref(n)) == status
    assert _route_call(lib, shape) == status
    cfg = B.router_cfg()
    assert lib.moe_route_backward(P, None, None, ctypes.byref(shape), ctypes.byref(cfg), P, P, None, None, None, P,
                                  None) == status


def test_route_refuses_arguments(lib):
    big = 1 << 30
    for kw in (dict(logits=None), dict(idx=None), dict(w=None), dict(logits=PAIR), dict(idx=PAIR), dict(bias=PAIR),
               dict(counts=P), dict(counts=P, tokens=P), dict(losses=P, ws=P, n=big),        # statistics: all or none
               dict(counts=P, tokens=P, losses=P),                                        # without a workspace
               dict(counts=P, tokens=P, losses=P, ws=ctypes.c_void_p((1 << 20) + 16), n=big),
               dict(counts=PAIR, tokens=P, losses=P, ws=P, n=big)):
        assert _route_call(lib, _shape(), **kw) == 1, kw
    assert _route_call(lib, _shape(dtype=1), logits=ODD) == 1
    assert _route_call(lib, _shape(S=2), counts=P, tokens=P, losses=P, ws=P, n=big) == 1     # S > 1 without offsets
    assert _route_call(lib, _shape(), counts=P, tokens=P, losses=P, ws=P, n=64) == 4
    assert _route_call(lib, _shape(E=8), cfg=B.router_cfg(n_group=3, topk_group=1)) == 1
    assert _route_call(lib, _shape(E=8, k=5), cfg=B.router_cfg(n_group=2, topk_group=1)) == 1
    assert _route_call(lib, _shape(E=8), cfg=B.router_cfg(n_group=4, topk_group=2, group_topn=3)) == 1
    assert _route_call(lib, _shape(E=64, ld=64), cfg=B.router_cfg(n_group=64, topk_group=2, group_topn=1)) == 2
    assert _route_call(lib, _shape(), cfg=B.RouterCfg(2, 1, 1.0, 1, 1, 1)) == 1
    assert _route_call(lib, _shape(T=0)) == 0
    cfg = B.router_cfg()

    def backward(logits=P, idx=P, dw=P, counts=None, tokens=None, dl=None, out=P, S=1, off=None):
        s = _shape(S=S)
        return lib.moe_route_backward(logits, None, off, ctypes.byref(s), ctypes.byref(cfg), idx, dw, counts, tokens, dl,
                                      out, None)
    for kw in (dict(logits=None), dict(idx=None), dict(dw=None), dict(out=None), dict(out=PAIR), dict(dl=P),
               dict(dl=P, counts=P), dict(dl=P, counts=P, tokens=P, S=2)):
        assert backward(**kw) == 1, kw
    assert lib.moe_bias_update(None, P, 1, 1, 8, 0.1, None) == 1
    assert lib.moe_bias_update(P, None, 1, 1, 8, 0.1, None) == 1
    assert lib.moe_bias_update(P, P, -1, 1, 8, 0.1, None) == 1
    assert lib.moe_bias_update(P, P, 1, 1, 1025, 0.1, None) == 2
    assert lib.moe_bias_update(P, P, 0, 1, 8, 0.1, None) == 0


def test_lists_refuse_arguments(lib):
    ptr = (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    bad = (ctypes.c_void_p * 2)(1 << 20, (1 << 21) + 1)
    null = (ctypes.c_void_p * 2)(1 << 20, None)
    n = (ctypes.c_int64 * 2)(4, 4)
    t = (ctypes.c_int32 * 2)(0, 1)
    big = 1 << 20

    def norm(p=ptr, n=n, t=t, count=2, kind=2, out=P, ws=P, size=big):
        return lib.moe_grad_norm(p, n, t, count, kind, out, ws, size, None)

    def clip(p=ptr, n=n, t=t, count=2, kind=2, most=1.0, out=P, ws=P, size=big):
        return lib.moe_clip_grads(p, n, t, count, kind, most, out, ws, size, None)
    for f in (norm, clip):
        for kw in (dict(p=None), dict(n=None), dict(t=None), dict(count=-1), dict(kind=3), dict(kind=-1), dict(out=None),
                   dict(out=PAIR), dict(ws=None), dict(ws=PAIR), dict(p=bad), dict(p=null),
                   dict(t=(ctypes.c_int32 * 2)(0, 7)), dict(n=(ctypes.c_int64 * 2)(4, -1))):
            assert f(**kw) == 1, kw
        assert f(size=64) == 4
        assert f(n=(ctypes.c_int64 * 2)(1 << 42, 1)) == 2
    for most in (-1.0, float("nan")):
        assert clip(most=most) == 1

    good = dict(b1=0.9, b2=0.99, eps=1e-8, most=0.0)

    def adamw(p=ptr, g=ptr, m=ptr, v=ptr, x=None, count=2, lr=P, step=P, ws=P, size=big, gt=t, **kw):
        a = {**good, **kw}
        cfg = B.AdamWCfg(a["b1"], a["b2"], a["eps"], 0.0, a["most"], 0)
        return lib.moe_adamw(p, t, g, gt, m, v, x, n, count, ctypes.byref(cfg), lr, step, None, ws, size, None)
    for kw in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(g=null), dict(m=null), dict(m=bad),
               dict(lr=None), dict(step=None), dict(step=PAIR), dict(ws=None), dict(gt=None), dict(b1=1.0), dict(b2=-0.1),
               dict(b2=float("nan")), dict(eps=-1.0), dict(most=-1.0), dict(x=bad), dict(count=-1)):
        assert adamw(**kw) == 1, kw
    assert adamw(size=64) == 4


def test_binding_refuses_types_and_layouts():
    x = torch.zeros((4, 8))
    idx = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((4, 2))
    with pytest.raises(ValueError):                       # not on a GPU
        B.moe_route(x, B.router_cfg(), idx, w)
    with pytest.raises(TypeError):
        B.moe_route(x.long(), B.router_cfg(), idx, w)
    m = torch.zeros((4, 8), device="meta")
    with pytest.raises(ValueError):
        B.moe_route(m[0], B.router_cfg(), idx, w)
    with pytest.raises(ValueError):
        B.moe_bias_update(x, x.int(), 0.1)
    with pytest.raises(ValueError):
        optim.clip_grad_norm_([], 1.0)
    with pytest.raises(ValueError):
        optim.clip_grad_norm_([x, x], 1.0)                # the same memory twice
    with pytest.raises(ValueError):
        optim.grad_norm([x])                              # not on a GPU
    with pytest.raises(ValueError):
        optim.AdamW([x]).step([x, x])
    assert optim.AdamW([x]).step() is None                # no gradients: nothing to do


def test_route_operators_on_meta_tensors():
    T, E, k = 12, 16, 3
    l = torch.empty((T, E), dtype=torch.bfloat16, device="meta", requires_grad=True)
    off = torch.empty((4,), dtype=torch.int32, device="meta")
    r = torch_ops.route(l, k, "sigmoid", seq_offsets=off)
    assert r.topk_idx.shape == (T, k) and r.topk_w.shape == (T, k) and r.counts.shape == (3, E)
    assert r.seq_tokens.shape == (5,) and r.topk_w.requires_grad and r.balance.requires_grad and not r.counts.requires_grad
    (r.topk_w.sum() + r.balance + r.z).backward()
    assert l.grad.shape == (T, E) and l.grad.dtype == torch.bfloat16
    H, I = 64, 32
    x = torch.empty((T, H), dtype=torch.bfloat16, device="meta", requires_grad=True)
    w1 = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device="meta", requires_grad=True)
    w2 = torch.empty((E, H, I), dtype=torch.bfloat16, device="meta", requires_grad=True)
    w = torch.empty((T, k), device="meta", requires_grad=True)
    y = torch_ops.moe_experts(x, r.topk_idx, w, w1, w2)
    y.backward(torch.empty_like(y))
    assert w.grad.shape == (T, k) and x.grad.shape == x.shape and w1.grad.shape == w1.shape and w2.grad.shape == w2.shape
    for bad in (dict(logits=l[0]), dict(logits=l.double()), dict(k=0), dict(k=E + 1), dict(score="relu"),
                dict(sel_bias=torch.empty((E + 1,), device="meta")), dict(token_mask=torch.empty((T,), device="meta")),
                dict(seq_offsets=torch.empty((4,), device="meta")),
                dict(seq_offsets=torch.empty((1,), dtype=torch.int32, device="meta"))):
        with pytest.raises((TypeError, ValueError)):
            torch_ops.route(**{**dict(logits=l, k=k), **bad})
