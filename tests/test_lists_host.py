"""Arguments of the list operators beyond a plain call's, on a host without a GPU."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

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


def test_numbers_in_place_of_tensors_are_refused():
    x = [torch.zeros((3,))]
    for f in (lambda: B.moe_adamw(x, x, x, x, 0.1, x[0], x[0], B.AdamWCfg()), lambda: B.moe_grad_norm(x, 0.0, x[0]),
              lambda: B.moe_bias_update([0.0], x[0], 0.1), lambda: B.moe_route([[0.0]], B.router_cfg(), x[0], x[0])):
        with pytest.raises(TypeError, match="torch tensor"):
            f()


class NoStream:
    cuda_stream = 0


@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
def test_operands_on_two_devices_are_refused(lib):
    def make(*shape, dtype=torch.float32, at=0):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{at}")
    kw = dict(stream=NoStream)
    with FakeTensorMode():
        i32 = torch.int32
        route = dict(topk_idx=((4, 2), i32), topk_w=((4, 2), torch.float32), sel_bias=((8,), torch.float32),
                     token_mask=((4,), torch.bool), seq_offsets=((2,), i32), counts=((1, 8), i32), seq_tokens=((3,), i32),
                     losses=((2,), torch.float32), ws=((4096,), torch.uint8))
        back = {n: v for n, v in route.items() if n in ("topk_idx", "token_mask", "seq_offsets", "counts", "seq_tokens")}
        back.update(dtopk_w=((4, 2), torch.float32), dlogits=((4, 8), torch.float32), dlosses=((2,), torch.float32))
        for f, operands in ((B.moe_route, route), (B.moe_route_backward, back)):
            for other in operands:
                args = {n: make(*s, dtype=t, at=int(n == other)) for n, (s, t) in operands.items()}
                with pytest.raises(ValueError, match="one device"):
                    f(make(4, 8), B.router_cfg(), **args, **kw)
        with pytest.raises(ValueError, match="one device"):
            B.moe_bias_update(make(8), make(1, 8, dtype=i32, at=1), 0.1, **kw)
        g, far = [make(5)], [make(5, at=1)]
        ws, norm = make(4096), make(1)
        for f in (lambda *a: B.moe_grad_norm(*a, **kw), lambda x, n, w: B.moe_clip_grads(x, 1.0, n, w, **kw)):
            for bad in ((far, norm, ws), (g, norm, make(4096, at=1)), (g, make(1, at=1), ws)):
                with pytest.raises(ValueError, match="one device"):
                    f(*bad)
        good = dict(params=g, grads=g, exp_avg=g, exp_avg_sq=g, lr=make(1), step=make(1, dtype=i32), ws=ws, cfg=B.AdamWCfg(),
                    masters=g, norm=norm, missed=make(1, dtype=i32))
        for name, bad in dict(params=far, grads=far, exp_avg=far, exp_avg_sq=far, masters=far, ws=make(4096, at=1),
                              step=make(1, dtype=i32, at=1), norm=make(1, at=1), missed=make(1, dtype=i32, at=1)).items():
            with pytest.raises(ValueError, match="one device"):
                B.moe_adamw(**{**good, name: bad}, **kw)
