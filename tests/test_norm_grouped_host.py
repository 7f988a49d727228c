"""The norm and the grouped products without a GPU: refusals of the C entry points, of the binding
and of the operators, and the operators' shapes and gradients on meta tensors."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import build as moe_build
from moe_expert_router_gb300 import torch_ops

P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.load()


def test_norm_refusals(lib):
    base = dict(T=4, H=128, ld_x=128, ld_r=128, eps=1e-6, dtype=1, w_dtype=0)
    p = 1 << 20

    def call(h=0, y=p + 16, codes=0, scales=0, x=p, residual=0, weight=p, rstd=0, **kw):
        s = B.NormShape(**(base | kw))
        return lib.moe_rms_norm(P(x), P(residual), P(weight), ctypes.byref(s), P(h), P(y), P(rstd), P(codes), P(scales), None)
    for kw in (dict(T=-1), dict(H=0), dict(ld_x=127), dict(ld_r=1), dict(eps=0.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(dtype=3), dict(dtype=-1), dict(w_dtype=2), dict(dtype=0, w_dtype=1), dict(x=0),
               dict(weight=0), dict(y=0), dict(codes=p), dict(scales=p), dict(h=p + 64), dict(x=p + 1), dict(weight=p + 2),
               dict(rstd=p + 2), dict(residual=p + 1), dict(codes=p + 8, scales=p), dict(codes=p, scales=p + 4),
               dict(residual=p, h=p + 16), dict(residual=p + 32, h=p, ld_x=136), dict(residual=p + 32, h=p + 32, ld_r=136),
               dict(codes=p, scales=p, y=p + 2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=16385, ld_x=16385, ld_r=16385), dict(T=2**31), dict(ld_x=2**31),
               dict(H=136, ld_x=136, ld_r=136, codes=p, scales=p)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, x=0, y=0, weight=0) == 0
    assert lib.moe_rms_norm(P(p), None, P(p), None, None, P(p), None, None, None, None) == INVALID

    def back(dy=p, dh=0, h=p, weight=p, rstd=p, dx=p, dweight=p, ws=p, n=1 << 30, **kw):
        s = B.NormShape(**(base | kw))
        return lib.moe_rms_norm_backward(P(dy), P(dh), P(h), P(weight), P(rstd), ctypes.byref(s), P(dx), P(dweight), P(ws), n, None)
    for kw in (dict(dy=0), dict(h=0), dict(weight=0), dict(rstd=0), dict(dx=0), dict(dweight=0), dict(ws=0), dict(ws=p + 8),
               dict(dy=p + 1), dict(dh=p + 1), dict(dweight=p + 2), dict(rstd=p + 1), dict(H=0), dict(dtype=7)):
        assert back(**kw) == INVALID, kw
    assert back(n=4 * 4 * 128 - 1) == WORKSPACE
    n = ctypes.c_size_t()
    assert lib.moe_rms_norm_workspace_size(4, 128, None) == INVALID
    assert lib.moe_rms_norm_workspace_size(-1, 128, ctypes.byref(n)) == INVALID
    assert lib.moe_rms_norm_workspace_size(4, 16385, ctypes.byref(n)) == UNSUPPORTED
    assert B.moe_rms_norm_workspace_size(0, 128) == 0
    assert B.moe_rms_norm_workspace_size(1 << 20, 128) >= 4 * 128 * (1 << 14)


def test_grouped_refusals(lib):
    base = dict(R=10, G=3, K=64, N=72, ld_x=64, ld_out=72, dtype=1, flags=0)
    p, need = 1 << 20, B.moe_grouped_workspace_size(3)

    def calls(x=p, w=p, offsets=p, out=p, ws=p, n=1 << 20, which=(0, 1, 2), **kw):
        s = B.GroupedShape(**(base | kw))
        ref = ctypes.byref(s)
        got = []
        if 0 in which:
            got.append(lib.moe_grouped_mm(P(x), P(w), P(offsets), ref, P(out), P(ws), n, None))
        if 1 in which:
            got.append(lib.moe_grouped_wgrad(P(x), P(w), P(offsets), ref, P(out), P(ws), n, None))
        if 2 in which and s.K % 128 == 0:
            got.append(lib.moe_grouped_mm_mx(P(x), P(x), P(w), P(w), P(offsets), ref, P(out), P(ws), n, None))
        return set(got)
    for k in (64, 128):
        for kw in (dict(R=-1), dict(G=0), dict(K=0), dict(N=0), dict(ld_x=56), dict(ld_out=64), dict(flags=2), dict(x=0),
                   dict(w=0), dict(offsets=0), dict(out=0), dict(x=p + 8), dict(w=p + 8), dict(out=p + 4), dict(offsets=p + 2),
                   dict(ws=0), dict(ws=p + 128)):
            assert calls(**(dict(K=k, ld_x=k) | kw)) == {INVALID}, kw
        for kw in (dict(G=1025), dict(K=k + 4, ld_x=k + 8), dict(N=76, ld_out=80), dict(ld_x=k + 4), dict(ld_out=76),
                   dict(dtype=0), dict(R=2**31 - 256), dict(G=1024, N=2**21, ld_out=2**21)):
            assert calls(**(dict(K=k, ld_x=k) | kw)) == {UNSUPPORTED}, kw
        assert calls(K=k, ld_x=k, n=need - 1) == {WORKSPACE}
    assert calls(which=(1,), flags=1) == {INVALID}
    mx = dict(K=128, ld_x=128)
    s = B.GroupedShape(**(base | mx | dict(flags=1)))
    assert lib.moe_grouped_mm_mx(P(p), P(p), P(p), P(p), P(p), ctypes.byref(s), P(p), P(p), 1 << 20, None) == INVALID
    for kw in (dict(dtype=2), dict(ld_x=136), dict(K=136, ld_x=136)):
        s = B.GroupedShape(**(base | mx | kw))
        assert lib.moe_grouped_mm_mx(P(p), P(p), P(p), P(p), P(p), ctypes.byref(s), P(p), P(p), 1 << 20, None) == UNSUPPORTED
    assert calls(R=0, x=0, out=0, which=(0,)) == {0}
    n = ctypes.c_size_t()
    assert lib.moe_grouped_workspace_size(0, ctypes.byref(n)) == INVALID
    assert lib.moe_grouped_workspace_size(3, None) == INVALID
    assert lib.moe_grouped_workspace_size(1025, ctypes.byref(n)) == UNSUPPORTED


def test_mx_dispatch_refusals(lib):
    p = 1 << 20
    s = B.shape(4, 256, 128, 8, 2, mxfp8=True)
    need = B.moe_workspace_size(s)

    def call(codes=p, scales=p, ws=p, n=need, s=s):
        a = lib.moe_mx_dispatch(P(codes), P(scales), ctypes.byref(s), P(ws), n, None)
        b = lib.moe_forward_mx_codes(P(codes), P(scales), P(p), P(p), P(p), P(p), P(p), P(p), ctypes.byref(s), P(p), P(ws), n, None)
        return {a, b}
    for kw in (dict(codes=0), dict(scales=0), dict(codes=p + 8), dict(scales=p + 4), dict(ws=0), dict(ws=p + 16)):
        assert call(**kw) == {INVALID}, kw
    assert call(n=need - 1) == {WORKSPACE}
    assert call(s=B.shape(4, 264, 128, 8, 2, mxfp8=True), n=1 << 30) == {UNSUPPORTED}
    assert call(s=B.shape(4, 256, 128, 8, 2), n=1 << 30) == {INVALID}
    assert call(s=B.shape(0, 256, 128, 8, 2, mxfp8=True)) <= {0}


class NoStream:
    cuda_stream = 0


def test_binding_refuses_host_tensors_and_numbers():
    moe_build.build()
    x, w = torch.zeros((4, 64)), torch.zeros((64,))
    m, o = torch.zeros((2, 72, 64)), torch.zeros((3,), dtype=torch.int32)
    for f in (lambda: B.moe_rms_norm(x, w, x, stream=NoStream), lambda: B.moe_rms_norm_backward(x, x, w, w, x, w, w, stream=NoStream),
              lambda: B.moe_grouped_mm(x, m, o, x, w, stream=NoStream), lambda: B.moe_grouped_wgrad(x, x, o, m, w, stream=NoStream),
              lambda: B.moe_grouped_mm_mx(x, x, m, m, o, x, w, stream=NoStream)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    for f in (lambda: B.moe_rms_norm([[0.0]], w, x), lambda: B.moe_grouped_mm(0.0, m, o, x, w),
              lambda: B.moe_rms_norm(0.0, w, x, stream=NoStream), lambda: B.moe_grouped_wgrad(3, x, o, m, w, stream=NoStream)):
        with pytest.raises(TypeError, match="torch tensor"):
            f()


def fake(*shape, dtype=BF16, stride=None):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t if stride is None else torch.empty_strided(shape, stride, dtype=dtype, device="cuda")


@pytest.mark.parametrize("error,match,call", [
    (TypeError, "x must be", lambda: B.moe_rms_norm(fake(4, 64, dtype=torch.float64), fake(64), fake(4, 64), stream=NoStream)),
    (ValueError, "two dimensions", lambda: B.moe_rms_norm(fake(4, 2, 64), fake(64), fake(4, 64), stream=NoStream)),
    (TypeError, "weight must be", lambda: B.moe_rms_norm(fake(4, 64), fake(64, dtype=torch.float16), fake(4, 64), stream=NoStream)),
    (ValueError, "weight must have", lambda: B.moe_rms_norm(fake(4, 64), fake(63), fake(4, 64), stream=NoStream)),
    (ValueError, "y must have", lambda: B.moe_rms_norm(fake(4, 64), fake(64), fake(4, 72), stream=NoStream)),
    (TypeError, "y must be", lambda: B.moe_rms_norm(fake(4, 64), fake(64), fake(4, 64, dtype=torch.float16), stream=NoStream)),
    (ValueError, "consecutive", lambda: B.moe_rms_norm(fake(4, 64, stride=(1, 4)), fake(64), fake(4, 64), stream=NoStream)),
    (ValueError, "overlap", lambda: B.moe_rms_norm(fake(4, 64, stride=(32, 1)), fake(64), fake(4, 64), stream=NoStream)),
    (ValueError, "y must be contiguous", lambda: B.moe_rms_norm(fake(4, 64), fake(64), fake(4, 64, stride=(72, 1)), stream=NoStream)),
    (ValueError, "out must have", lambda: B.moe_grouped_mm(fake(4, 64), fake(2, 72, 64), fake(3, dtype=torch.int32), fake(4, 64), fake(9), stream=NoStream)),
    (ValueError, "fits", lambda: B.moe_grouped_mm(fake(4, 64), fake(2, 72, 64), fake(3, dtype=torch.int32), fake(4, 72), fake(9), transposed=True, stream=NoStream)),
    (TypeError, "x must be", lambda: B.moe_grouped_mm(fake(4, 64, dtype=torch.float32), fake(2, 72, 64), fake(3, dtype=torch.int32), fake(4, 72), fake(9), stream=NoStream)),
    (TypeError, "w must be", lambda: B.moe_grouped_mm(fake(4, 64), fake(2, 72, 64, dtype=torch.float16), fake(3, dtype=torch.int32), fake(4, 72), fake(9), stream=NoStream)),
    (ValueError, "offsets must have", lambda: B.moe_grouped_mm(fake(4, 64), fake(2, 72, 64), fake(2, dtype=torch.int32), fake(4, 72), fake(9), stream=NoStream)),
    (TypeError, "offsets must be", lambda: B.moe_grouped_mm(fake(4, 64), fake(2, 72, 64), fake(3, dtype=torch.int64), fake(4, 72), fake(9), stream=NoStream)),
    (ValueError, "b must have", lambda: B.moe_grouped_wgrad(fake(4, 64), fake(5, 72), fake(3, dtype=torch.int32), fake(2, 64, 72), fake(9), stream=NoStream)),
    (ValueError, "fits", lambda: B.moe_grouped_wgrad(fake(4, 64), fake(4, 72), fake(3, dtype=torch.int32), fake(2, 72, 64), fake(9), stream=NoStream)),
])
def test_binding_refuses_types_and_shapes(error, match, call):
    moe_build.build()
    with FakeTensorMode():
        with pytest.raises(error, match=match):
            call()


def test_operators_on_meta_tensors():
    m = lambda *s, dtype=BF16, grad=False: torch.empty(s, dtype=dtype, device="meta", requires_grad=grad)  # noqa: E731
    x, r, w = m(10, 256, grad=True), m(10, 256, grad=True), m(256, dtype=torch.float32, grad=True)
    y, h = torch_ops.rms_norm(x, w, residual=r)
    assert y.shape == h.shape == x.shape
    (y + h).sum().backward()
    assert x.grad.shape == r.grad.shape == x.shape and w.grad.shape == (256,) and w.grad.dtype == torch.float32
    assert torch_ops.rms_norm(x, w).shape == x.shape
    y, h, c, s = torch_ops.rms_norm_mx(m(10, 256), m(256))
    assert h.shape == (0, 256) and c.shape == (10, 256) and s.shape == (2, 12, 4)
    g, o = m(3, 72, 256, grad=True), m(4, dtype=torch.int32)
    out = torch_ops.grouped_mm(x, g, o)
    assert out.shape == (10, 72)
    out.sum().backward()
    assert g.grad.shape == g.shape
    assert torch_ops.grouped_mm(m(10, 72), m(3, 72, 256), o, transposed=True).shape == (10, 256)
    y = torch.ops.moe_gb300.forward_mx_codes(c, s, m(10, 2, dtype=torch.int32), m(10, 2, dtype=torch.float32),
                                            m(4, 256, 256, dtype=torch.uint8), m(2, 4, 256, 4, dtype=torch.uint8),
                                            m(4, 256, 128, dtype=torch.uint8), m(1, 4, 256, 4, dtype=torch.uint8))
    assert y.shape == (10, 256) and y.dtype == BF16
    for error, f in ((ValueError, lambda: torch_ops.rms_norm(m(10, 256), m(255))),
                     (TypeError, lambda: torch_ops.rms_norm(m(10, 256), m(256, dtype=torch.float16))),
                     (ValueError, lambda: torch_ops.rms_norm(m(10, 256), m(256), eps=0.0)),
                     (ValueError, lambda: torch_ops.rms_norm(m(10, 16392), m(16392))),
                     (ValueError, lambda: torch_ops.rms_norm(m(10, 256), m(256), m(11, 256))),
                     (ValueError, lambda: torch_ops.rms_norm_mx(m(10, 200), m(200))),
                     (ValueError, lambda: torch_ops.grouped_mm(m(10, 64), m(3, 72, 256), o)),
                     (ValueError, lambda: torch_ops.grouped_mm(m(10, 64), m(3, 12, 64), o)),
                     (TypeError, lambda: torch_ops.grouped_mm(m(10, 64, dtype=torch.float32), m(3, 72, 64), o)),
                     (ValueError, lambda: torch_ops.grouped_mm(m(10, 64), m(3, 72, 64), m(3, dtype=torch.int32)))):
        with pytest.raises(error):
            f()
