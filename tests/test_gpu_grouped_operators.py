"""The differentiable grouped product where its offsets are bad, and operands that are views at odd places."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import torch_ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def whole(gen, *shape, dtype=BF16):
    return torch.randint(-2, 3, shape, generator=gen, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R", [10, 700])
@pytest.mark.parametrize("last", [-3, 701])
def test_bad_offsets_are_seen(dtype, R, last):
    """Offsets that decrease, or leave the rows: everything that comes out is NaN, and the call's error word
    says why. (Few rows and many take kernels of their own.)"""
    gen = torch.Generator(DEV).manual_seed(0)
    bad = torch.tensor([0, 5, 7, last if last < 0 else R + 1], dtype=torch.int32, device=DEV)
    good = torch.tensor([0, 5, 7, R], dtype=torch.int32, device=DEV)
    for transposed in (False, True):
        for complete in (False, True):
            x = whole(gen, R, 64, dtype=dtype).requires_grad_()
            w = (whole(gen, 3, 64, 72, dtype=dtype) if transposed else whole(gen, 3, 72, 64, dtype=dtype)).requires_grad_()
            out, word = torch_ops.grouped_mm(x, w, bad, transposed=transposed, complete=complete, errors=True)
            assert word.item() == B.DEVERR_BAD_OFFSETS
            assert torch.isnan(out).all()
            out.backward(torch.ones_like(out))
            assert torch.isnan(x.grad).all() and torch.isnan(w.grad).all()
            assert torch.isnan(torch_ops.grouped_mm(x, w, bad, transposed=transposed, complete=complete)).all()
            x.grad = w.grad = None
            out, word = torch_ops.grouped_mm(x, w, good, transposed=transposed, complete=complete, errors=True)
            assert word.item() == 0 and torch.isfinite(out).all()
            same = torch_ops.grouped_mm(x, w, good, transposed=transposed, complete=complete)
            assert torch.equal(out, same)
            grads = torch.autograd.grad(out, (x, w), torch.ones_like(out))
            for a, b in zip(grads, torch.autograd.grad(same, (x, w), torch.ones_like(same))):
                assert torch.equal(a, b) and torch.isfinite(a).all()


def test_bad_offsets_through_the_binding():
    """nan_on_bad fills all of out, and nothing between its rows."""
    gen = torch.Generator(DEV).manual_seed(1)
    for R in (10, 700):
        bad = torch.tensor([0, 5, 3, R], dtype=torch.int32, device=DEV)
        x, w = whole(gen, R, 64), whole(gen, 3, 72, 64)
        buf, ws = torch.full((R, 80), 77.0, dtype=BF16, device=DEV), B.grouped_workspace(3)
        B.moe_grouped_mm(x, w, bad, buf[:, :72], ws, nan_on_bad=True)
        assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS
        assert torch.isnan(buf[:, :72]).all() and (buf[:, 72:] == 77).all()
        dw = torch.full_like(w, 77.0)
        B.moe_grouped_wgrad(whole(gen, R, 72), x, bad, dw, ws, nan_on_bad=True)
        assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and torch.isnan(dw).all()
        good, out = torch.tensor([2, 5, 5, R], dtype=torch.int32, device=DEV), torch.full((R, 72), 77.0, dtype=BF16, device=DEV)
        a, b = out.clone(), out.clone()
        B.moe_grouped_mm(x, w, good, a, ws, nan_on_bad=True)
        B.moe_grouped_mm(x, w, good, b, ws)
        assert torch.equal(a, b) and (a[:2] == 77).all()


def test_error_word_of_a_captured_call():
    gen = torch.Generator(DEV).manual_seed(2)
    x, w = whole(gen, 300, 64), whole(gen, 3, 72, 64)
    offsets = torch.tensor([0, 5, 7, 300], dtype=torch.int32, device=DEV)
    want = torch_ops.grouped_mm(x, w, offsets, complete=True)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch_ops.grouped_mm(x, w, offsets, complete=True)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out, word = torch_ops.grouped_mm(x, w, offsets, complete=True, errors=True)
    good = offsets.clone()
    for bad in (False, True, False):
        offsets.copy_(good)
        if bad:
            offsets[2] = 400
        graph.replay()
        torch.cuda.synchronize()
        assert word.item() == (B.DEVERR_BAD_OFFSETS if bad else 0)
        assert torch.isnan(out).all() if bad else torch.equal(out, want)


def at_odd_place(t, by):
    """The same values as a dense view `by` elements into a flat buffer."""
    flat = torch.zeros((t.numel() + by,), dtype=t.dtype, device=DEV)
    out = flat[by:].view(t.shape)
    out.copy_(t)
    return out


def test_matrices_at_odd_places():
    gen = torch.Generator(DEV).manual_seed(3)
    x, dy = whole(gen, 190, 136), whole(gen, 190, 72)
    o = torch.tensor([2, 50, 50, 181], dtype=torch.int32, device=DEV)
    for transposed in (False, True):
        w = whole(gen, 3, 136, 72) if transposed else whole(gen, 3, 72, 136)
        got = []
        for by in (0, 1, 4):
            xs, ws = x.clone().requires_grad_(), at_odd_place(w, by).requires_grad_()
            out = torch_ops.grouped_mm(xs, ws, o, transposed=transposed)
            got.append((out, *torch.autograd.grad(out, (xs, ws), at_odd_place(dy, by))))
        for other in got[1:]:
            for a, b in zip(got[0], other):
                assert torch.equal(a, b)


def test_norm_weights_at_odd_places():
    gen = torch.Generator(DEV).manual_seed(4)
    T, H = 9, 256
    x, r = torch.randn((T, H), generator=gen, device=DEV).to(BF16), torch.randn((T, H), generator=gen, device=DEV).to(BF16)
    for w in (torch.randn((H,), generator=gen, device=DEV), torch.randn((H,), generator=gen, device=DEV).to(BF16)):
        want = torch_ops.rms_norm_mx(x, w, r)
        got = torch_ops.rms_norm_mx(x, at_odd_place(w, 3), r)
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b)
        assert torch.equal(got[3][:, :T], want[3][:, :T])
        assert torch.equal(torch_ops.rms_norm(x, at_odd_place(w, 3)), torch_ops.rms_norm(x, w))


def test_codes_at_odd_places():
    gen = torch.Generator(DEV).manual_seed(5)
    T, H, I, E, k = 9, 256, 128, 4, 2
    x = torch.randn((T, H), generator=gen, device=DEV).to(BF16)
    q = []
    for shape in ((E, 2 * I, H), (E, H, I)):
        m = torch.randn(shape, generator=gen, device=DEV).to(BF16)
        q += [torch.empty(shape, dtype=torch.uint8, device=DEV), B.mx_scales_empty(shape, DEV)]
        B.moe_mx_quantize(m, *q[-2:])
    idx = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1)[1].int()
    w = torch.rand((T, k), generator=gen, device=DEV)
    _, _, codes, scales = torch_ops.rms_norm_mx(x, torch.ones((H,), device=DEV))
    want = torch.ops.moe_gb300.forward_mx_codes(codes, scales, idx, w, *q)
    got = torch.ops.moe_gb300.forward_mx_codes(at_odd_place(codes, 5), at_odd_place(scales, 4), idx, w, *q)
    assert torch.equal(got, want)
