"""What the norm's and the grouped products' C entry points refuse beyond single arguments, without a GPU."""
import ctypes

import pytest
import torch

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import build as moe_build
from moe_expert_router_gb300 import torch_ops

P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.load()


def test_norm_outputs_over_rows_apart(lib):
    """y in the place of x or of the residual, whose rows lie apart: its dense rows would lie over other rows."""
    p = 1 << 20

    def call(T=4, ld_x=128, ld_r=128, x=p, residual=0, h=0, y=p + (1 << 19)):
        s = B.NormShape(T=T, H=128, ld_x=ld_x, ld_r=ld_r, eps=1e-6, dtype=1, w_dtype=0)
        return lib.moe_rms_norm(P(x), P(residual), P(p + 64), ctypes.byref(s), P(h), P(y), None, None, None, None)
    far = p + (1 << 18)
    for kw in (dict(ld_x=136, y=p), dict(residual=far, ld_r=136, y=far), dict(residual=far, ld_r=129, y=far, h=p),
               dict(residual=far, ld_x=256, y=p, h=far), dict(T=2, ld_x=136, y=p)):
        assert call(**kw) == INVALID, kw


def test_grouped_sizes_at_the_end_of_32_bits(lib):
    """Sizes whose counters in the kernels would pass 2^31 are refused before a launch: the few-row kernel
    counts up to 2048 columns past K."""
    p = 1 << 20

    def calls(R=4, G=1, K=64, N=64):
        s = B.GroupedShape(R=R, G=G, K=K, N=N, ld_x=K, ld_out=N, dtype=1, flags=0)
        ref, n = ctypes.byref(s), 1 << 20
        got = {lib.moe_grouped_mm(P(p), P(p), P(p), ref, P(p), P(p), n, None),
               lib.moe_grouped_wgrad(P(p), P(p), P(p), ref, P(p), P(p), n, None)}
        if K % 128 == 0:
            got.add(lib.moe_grouped_mm_mx(P(p), P(p), P(p), P(p), P(p), ref, P(p), P(p), n, None))
        return got
    end = 2**31
    for kw in (dict(K=end - 512), dict(K=end - 4096), dict(N=end - 512), dict(N=end - 4096), dict(G=8, K=end // 8 - 8),
               dict(G=512, N=end // 512 - 8), dict(K=end - 264, N=8), dict(R=end - 264, N=2**16, K=8)):
        assert calls(**kw) == {UNSUPPORTED}, kw


def test_grouped_flags(lib):
    """NaN for bad offsets is a flag of the 16-bit products; others are refused."""
    p = 1 << 20

    def call(f, flags):
        s = B.GroupedShape(R=10, G=3, K=128, N=72, ld_x=128, ld_out=72, dtype=1, flags=flags)
        args = [P(p)] * (5 if f == "moe_grouped_mm_mx" else 3)
        return getattr(lib, f)(*args, ctypes.byref(s), P(p), P(p), 8, None)
    for f, flags in (("moe_grouped_mm", 8), ("moe_grouped_mm", 6), ("moe_grouped_wgrad", 5), ("moe_grouped_wgrad", 2),
                     ("moe_grouped_mm_mx", 4)):
        assert call(f, flags) == INVALID
    for f, flags in (("moe_grouped_mm", 4), ("moe_grouped_mm", 5), ("moe_grouped_wgrad", 4), ("moe_grouped_mm_mx", 0)):
        assert call(f, flags) == WORKSPACE                  # the flags are taken: what fails is the workspace's size


def test_checked_product_on_meta_tensors():
    m = lambda *s, dtype=torch.bfloat16, grad=False: torch.empty(s, dtype=dtype, device="meta", requires_grad=grad)  # noqa: E731
    x, w = m(10, 256, grad=True), m(3, 72, 256, grad=True)
    out, word = torch_ops.grouped_mm(x, w, m(4, dtype=torch.int32), errors=True)
    assert out.shape == (10, 72) and word.shape == (1,) and word.dtype == torch.int32 and not word.requires_grad
    out.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
