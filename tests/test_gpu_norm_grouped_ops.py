"""The norm and the grouped products as a model uses them: the operators and their gradients, experts
built from them in front of and beside the layer's own path, and what the binding refuses."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from moe_expert_router_gb300 import torch_ops
from moe_expert_router_gb300.mx_cache import MxWeightCache

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def randn(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def test_norm_operator_gradients():
    gen = torch.Generator(DEV).manual_seed(0)
    T, H = 77, 640
    x, r = randn(gen, T, H).requires_grad_(), randn(gen, T, H).requires_grad_()
    w = (1 + 0.1 * torch.randn((H,), generator=gen, device=DEV)).requires_grad_()
    dy, dh = randn(gen, T, H), randn(gen, T, H)
    y, h = torch_ops.rms_norm(x, w, r, eps=1e-5)
    torch.autograd.backward((y, h), (dy, dh))
    rstd, y1, h1 = torch.empty((T,), device=DEV), torch.empty_like(x), torch.empty_like(x)
    B.moe_rms_norm(x.detach(), w.detach(), y1, 1e-5, residual=r.detach(), h=h1, rstd=rstd)
    dx, dw = torch.empty_like(dy), torch.empty((H,), device=DEV)
    B.moe_rms_norm_backward(dy, h1, w.detach(), rstd, dx, dw, B.rms_norm_scratch(T, H, dx), dh=dh)
    assert torch.equal(y, y1) and torch.equal(h, h1)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx) and torch.equal(w.grad, dw)
    # the norm alone, the stream alone, a transposed input and an expanded gradient
    for t in (x, r, w):
        t.grad = None
    torch_ops.rms_norm(x, w, r)[1].backward(dh)
    assert torch.equal(x.grad, dh) and torch.equal(r.grad, dh) and w.grad is None
    x2 = randn(gen, H, T).t().requires_grad_()
    y = torch_ops.rms_norm(x2, w)
    y.sum().backward()                                      # dy is one number, expanded
    y1, rs = torch.empty_like(y), torch.empty((T,), device=DEV)
    B.moe_rms_norm(x2.detach().contiguous(), w.detach(), y1, rstd=rs)
    assert torch.equal(y, y1)
    B.moe_rms_norm_backward(torch.ones_like(y1), x2.detach().contiguous(), w.detach(), rs, dx, dw, B.rms_norm_scratch(T, H, dx))
    assert torch.equal(x2.grad, dx) and torch.equal(w.grad, dw)


def test_captured_forward_and_backward():
    gen = torch.Generator(DEV).manual_seed(1)
    x, w = randn(gen, 64, 256).requires_grad_(), torch.ones((256,), device=DEV, requires_grad=True)
    m = randn(gen, 2, 128, 256, scale=0.1).requires_grad_()
    o = torch.tensor([0, 20, 64], dtype=torch.int32, device=DEV)
    grads = lambda: torch.autograd.grad(torch_ops.grouped_mm(torch_ops.rms_norm(x, w), m, o, complete=True).float().square().sum(), (x, w, m))  # noqa: E731
    want = grads()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        grads()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = grads()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_operator_gradients(dtype):
    gen = torch.Generator(DEV).manual_seed(2)
    o = torch.tensor([2, 50, 50, 181], dtype=torch.int32, device=DEV)
    x = torch.randint(-2, 3, (190, 136), generator=gen, device=DEV).to(dtype)
    w = torch.randint(-2, 3, (3, 72, 136), generator=gen, device=DEV).to(dtype)
    dy = torch.randint(-2, 3, (190, 72), generator=gen, device=DEV).to(dtype)
    cuts = [(2, 50), (50, 50), (50, 181)]
    for transposed in (False, True):
        xs = torch.nn.functional.pad(x, (3, 2))[:, 3:-2].requires_grad_()     # rows at odd places: copied
        ws = (w.transpose(1, 2).contiguous() if transposed else w).clone().requires_grad_()
        out = torch_ops.grouped_mm(xs, ws, o, transposed=transposed)
        out.backward(dy)
        y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)
        for g, (a, b) in enumerate(cuts):
            y[a:b] = (x[a:b].double() @ w[g].double().t()).to(dtype)
            dx[a:b] = (dy[a:b].double() @ w[g].double()).to(dtype)
            dw[g] = (dy[a:b].double().t() @ x[a:b].double()).to(dtype)
        assert torch.equal(out, y) and torch.equal(xs.grad, dx)
        assert torch.equal(ws.grad, dw.transpose(1, 2) if transposed else dw)


def routed(gen, T, E, k, shp, ws):
    """A routing, its metadata in ws, and the groups' offsets and rows' tokens."""
    idx = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1)[1].int()
    w = torch.rand((T, k), generator=gen, device=DEV)
    B.moe_routing_metadata(idx, shp, ws)
    lay = B.moe_workspace_layout(shp)
    offsets = ws[lay.offsets:lay.offsets + 4 * (E + 1)].view(torch.int32)
    slot = ws[lay.perm_slot:lay.perm_slot + 4 * T * k].view(torch.int32).clone()
    return idx, w, offsets, slot


def test_experts_from_grouped_products_equal_the_layer():
    """norm -> dispatch -> grouped product -> SwiGLU -> grouped product -> combine against the expert
    path on the same normed rows, and the gradients of both. The two round their hidden values in
    other places (h to bf16 before the SwiGLU here), so they agree to a few bf16 steps: the error of
    each is under the path's own bound, 1e-2 of the norm."""
    gen = torch.Generator(DEV).manual_seed(3)
    T, H, I, E, k = 300, 256, 136, 8, 2
    shp = B.shape(T, H, I, E, k)
    ws = B.new_workspace(shp, DEV)
    idx, w, offsets, slot = routed(gen, T, E, k, shp, ws)
    x, r = randn(gen, T, H), randn(gen, T, H)
    gain = (1 + 0.1 * torch.randn((H,), generator=gen, device=DEV))
    w1, w2 = randn(gen, E, 2 * I, H, scale=H ** -0.5), randn(gen, E, H, I, scale=I ** -0.5)
    dy = randn(gen, T, H)

    def grads(experts):
        ts = [t.clone().requires_grad_() for t in (x, r, gain, w1, w2, w)]
        y, h = torch_ops.rms_norm(ts[0], ts[2], ts[1])
        out = h + experts(y, *ts[3:])
        return [out] + list(torch.autograd.grad(out, ts, dy))

    def from_products(n, w1, w2, w):
        token = (slot // k).long()
        g = torch_ops.grouped_mm(n[token], w1, offsets, complete=True).float()
        a = (torch.nn.functional.silu(g[:, :I]) * g[:, I:]).to(BF16)
        o = torch_ops.grouped_mm(a, w2, offsets, complete=True).float() * w.flatten()[slot.long()][:, None]
        return torch.zeros((T, H), device=DEV).index_add(0, token, o).to(BF16)
    a, b = grads(from_products), grads(lambda n, w1, w2, w: torch_ops.moe_experts(n, idx, w, w1, w2))
    for name, p, q in zip(("y", "dx", "dr", "dgain", "dw1", "dw2", "dw"), a, b):
        rel = ((p.double() - q.double()).norm() / q.double().norm()).item()
        assert rel < 2e-2, (name, rel)
    # the dispatch's own rows are those products' operands
    rows = torch.empty((T * k, H), dtype=BF16, device=DEV)
    B.moe_dispatch_rows(x, shp, rows, ws)
    out, out2 = torch.empty((T * k, 2 * I), dtype=BF16, device=DEV), torch.empty((T * k, 2 * I), dtype=BF16, device=DEV)
    gw = B.grouped_workspace(E, DEV)
    B.moe_grouped_mm(rows, w1, offsets, out, gw)
    B.moe_grouped_mm(x[(slot // k).long()], w1, offsets, out2, gw)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 128, 4, 2), (7, 256, 128, 8, 3), (130, 1152, 256, 16, 4), (999, 256, 128, 4, 1)])
def test_codes_of_the_norm_through_the_mxfp8_path(T, H, I, E, k):
    """norm with codes -> forward_mx_codes gives the bits of norm -> forward_mx."""
    gen = torch.Generator(DEV).manual_seed(T)
    x, r, gain = randn(gen, T, H), randn(gen, T, H), torch.ones((H,), device=DEV)
    w1, w2 = randn(gen, E, 2 * I, H, scale=H ** -0.5), randn(gen, E, H, I, scale=I ** -0.5)
    cache = MxWeightCache()
    q = [*cache.get(w1), *cache.get(w2)]
    idx = torch.rand((T, E), generator=gen, device=DEV).topk(k, dim=1)[1].int()
    idx[T // 2, 0] = -1                                     # a slot left over
    w = torch.rand((T, k), generator=gen, device=DEV)
    y, h, codes, scales = torch_ops.rms_norm_mx(x, gain, r)
    ops = torch.ops.moe_gb300
    assert torch.equal(ops.forward_mx_codes(codes, scales, idx, w, *q), ops.forward_mx(y, idx, w, *q))
    # stage by stage: the dispatched codes and words
    shp = B.shape(T, H, I, E, k, mxfp8=True)
    lay = B.moe_workspace_layout(shp)
    got = []
    for codes_in in (True, False):
        ws = B.new_workspace(shp, DEV)
        ws[256:].fill_(0x5a)
        B.moe_routing_metadata(idx, shp, ws)
        B.moe_mx_dispatch(codes, scales, shp, ws) if codes_in else B.moe_mx_quantize_dispatch(y, shp, ws)
        got.append((ws[lay.x_codes:lay.x_codes + T * k * H].clone(),
                    ws[lay.x_scales:lay.x_scales + (T * k + 3) // 4 * 4 * H // 32].clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    # and straight into a grouped product, rows in token order
    o = torch.tensor([0, T // 3, T], dtype=torch.int32, device=DEV)
    m = randn(gen, 2, 72, H)
    mc, ms = torch.empty((2, 72, H), dtype=torch.uint8, device=DEV), B.mx_scales_empty((2, 72, H), DEV)
    B.moe_mx_quantize(m, mc, ms)
    a, gw = torch.empty((T, 72), dtype=BF16, device=DEV), B.grouped_workspace(2, DEV)
    B.moe_grouped_mm_mx(codes, scales, mc, ms, o, a, gw)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    B.moe_mx_quantize(y, c2, s2)
    b = torch.empty_like(a)
    B.moe_grouped_mm_mx(c2, s2, mc, ms, o, b, gw)
    assert torch.equal(a, b)


def test_norm_mxfp8_of_rows_at_odd_places():
    gen = torch.Generator(DEV).manual_seed(8)
    for dtype in (BF16, F16, torch.float32):
        for T, H in ((3, 128), (5, 1152), (2, 8192), (2, 9088)):
            x, r = randn(gen, T, H + 5, dtype=dtype)[:, :H], randn(gen, T, H + 3, dtype=dtype)[:, 2:H + 2]
            w = randn(gen, H, dtype=dtype)
            got = torch_ops.rms_norm_mx(x, w, r)
            want = torch_ops.rms_norm_mx(x.contiguous(), w, r.contiguous())
            for a, b in zip(got[:3], want[:3]):
                assert torch.equal(a, b)
            assert torch.equal(got[3].view(H // 128, -1, 4)[:, :T], want[3].view(H // 128, -1, 4)[:, :T])


def test_shared_memory_is_refused():
    buf = torch.zeros((64, 512), dtype=BF16, device=DEV)
    w, f = torch.ones((128,), device=DEV), torch.empty((64,), device=DEV)
    x, y = buf[:, :128], torch.empty((64, 128), dtype=BF16, device=DEV)
    flat = torch.zeros((64 * 128 + 8,), dtype=BF16, device=DEV)
    a, b = flat[:-8].view(64, 128), flat[8:].view(64, 128)
    same = pytest.raises(ValueError, match="the same memory")
    with same:
        B.moe_rms_norm(a, w, b)
    with same:
        B.moe_rms_norm(x, w, y, residual=x, h=y)
    with same:
        B.moe_rms_norm(x, flat[:256].view(torch.float32), flat[:8192].view(64, 128))
    with same:
        B.moe_rms_norm(a, w, y, codes=flat[:4096].view(torch.uint8).view(64, 128), scales=B.mx_scales_empty((64, 128), DEV))
    ws = B.rms_norm_scratch(64, 128, x)
    with same:
        B.moe_rms_norm_backward(y, a, w, f, b, torch.empty_like(w), ws)
    with same:
        B.moe_rms_norm_backward(y, a, w, f, a, torch.empty_like(w), ws)
    with same:
        B.moe_rms_norm_backward(y, a, w, f, torch.empty_like(y), w, ws)
    o, gw = torch.tensor([0, 64], dtype=torch.int32, device=DEV), B.grouped_workspace(1, DEV)
    m = torch.zeros((1, 128, 128), dtype=BF16, device=DEV)
    with same:
        B.moe_grouped_mm(a, m, o, b, gw)
    with same:
        B.moe_grouped_mm(a, m, o, m[0, :64], gw)
    with same:
        B.moe_grouped_mm(buf[:, :128], m, o, buf[:, 64:192], gw)
    with same:
        B.moe_grouped_wgrad(m[0], m[0], o, m, gw)
    two = torch.zeros((64, 128), dtype=BF16)
    with pytest.raises(ValueError):
        B.moe_grouped_mm(a, two.view(1, 64, 128), o, y, gw)


def test_written_operands_count_a_version():
    x, w, y = torch.ones((4, 64), dtype=BF16, device=DEV), torch.ones((64,), device=DEV), torch.empty((4, 64), dtype=BF16, device=DEV)
    m, o, gw = torch.ones((1, 64, 64), dtype=BF16, device=DEV), torch.tensor([0, 4], dtype=torch.int32, device=DEV), B.grouped_workspace(1, DEV)
    h = torch.empty_like(y)
    before = (y._version, h._version, m._version, x._version)
    B.moe_rms_norm(x, w, y, residual=x, h=h)
    B.moe_grouped_mm(x, m, o, y, gw)
    B.moe_grouped_wgrad(x, x, o, m, gw)
    assert (y._version, h._version, m._version, x._version) == (before[0] + 2, before[1] + 1, before[2] + 1, before[3])
