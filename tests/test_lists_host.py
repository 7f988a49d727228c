"""Arguments of the list operators beyond a plain call's, on a host without a GPU."""
import ctypes

import pytest

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import build as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return B.load()


def test_adamw_configuration(lib):
    assert B.AdamWCfg(0.9, 0.999).beta2 == 0.999          # 64 bits: 1 - beta is taken there
    ptr = (ctypes.c_void_p * 1)(1 << 20)
    n, t, p = (ctypes.c_int64 * 1)(4), (ctypes.c_int32 * 1)(0), ctypes.c_void_p(1 << 20)

    def adamw(**kw):
        cfg = B.AdamWCfg(0.9, 0.999, 1e-8)
        for name, v in kw.items():
            setattr(cfg, name, v)
        return lib.moe_adamw(ptr, t, ptr, t, ptr, ptr, None, n, 1, ctypes.byref(cfg), p, p, None, p, 1 << 20, None)
    for kw in (dict(missed=(1 << 20) + 2), dict(beta1=1.0), dict(beta2=-1e-9), dict(beta2=float("nan"))):
        assert adamw(**kw) == 1, kw
