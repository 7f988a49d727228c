"""What the norm's and the grouped products' C entry points refuse beyond single arguments, without a GPU."""
import ctypes

import pytest

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import build as moe_build

P = ctypes.c_void_p
INVALID, UNSUPPORTED = 1, 2


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
