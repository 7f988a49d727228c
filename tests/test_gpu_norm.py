"""The norm in front of the layer against its formulas in 64 bits: types, widths, strides, memory
in place, its MXFP8 form, gradients.

y is the exact value rounded once: equal to the 64-bit result rounded once (fp32: two roundings to
48 bits come before the last one, so a relative 2^-24 (1 + 2^-20)). The gradients' bounds follow from
their roundings, each at most 2^-24 of a magnitude: a gradient dx takes four to z and g, two to the
bracket, one to the stream's gradient, and the mean of the row at most 4 (vectors) x 8 + 10 (the
threads) additions in a row and three roundings of each product; dweight at most 64 + 32 additions in
a row and three roundings of each product. Half a step of the type is added for the last rounding."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def rounded(v, dtype):
    """64-bit values rounded once to `dtype` (a conversion would round twice, by way of fp32)."""
    f = v.float()
    if dtype == F32:
        return f
    low = v - f.double()
    bits = f.view(torch.int32)
    odd = torch.where((bits & 1 == 0) & (low != 0), torch.sign(low * f.double()).int(), 0)
    return (bits + odd).view(F32).to(dtype)


def wide(gen, T, H, dtype, pad, scale=1.0):
    return torch.randn((T, H + pad), generator=gen, device=DEV).mul_(scale).to(dtype)[:, :H]


def reference(x, residual, weight, eps):
    h = x if residual is None else rounded(x.double() + residual.double(), x.dtype)
    h64 = h.double()
    rstd = 1.0 / torch.sqrt(h64.square().mean(1, keepdim=True) + eps)
    return h, h64 * rstd * weight.double(), rstd[:, 0]


def half_step(v, dtype):
    return torch.finfo(dtype).eps / 2 * v.abs().clamp(min=torch.finfo(dtype).smallest_normal)


def assert_y(y, exact):
    if y.dtype == F32:
        assert ((y.double() - exact).abs() <= exact.abs() * U * (1 + 2.0 ** -20) + 2.0 ** -149).all()
    else:
        assert torch.equal(y, rounded(exact, y.dtype))


SIZES = [(1, 1), (3, 7), (1, 8), (5, 24), (2, 31), (9, 128), (33, 129), (1, 256), (7, 257), (300, 512), (17, 1000),
         (5, 1003), (8, 1024), (2, 1032), (9, 2048), (3, 4096), (1, 7168), (6, 7168), (2, 8200), (2, 8191), (3, 16384),
         (2, 16383), (2, 16376)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F32), (BF16, BF16), (F16, F32), (F16, F16), (F32, F32)])
def test_forward_and_backward(T, H, dtype, w_dtype):
    gen = torch.Generator(DEV).manual_seed(1000 * T + H)
    for residual, pad in ((True, 0), (False, 0), (True, 8), (False, 5)):
        x = wide(gen, T, H, dtype, pad, 3.0)
        r = wide(gen, T, H, dtype, pad + (3 if pad == 5 else 0)) if residual else None
        w = (1.0 + 0.3 * torch.randn((H,), generator=gen, device=DEV)).to(w_dtype)
        y = torch.full((T, H), 99.0, dtype=dtype, device=DEV)
        h = torch.full_like(y, 99.0) if residual else None
        rstd = torch.full((T,), 99.0, device=DEV)
        B.moe_rms_norm(x, w, y, 1e-6, residual=r, h=h, rstd=rstd)
        h_ref, exact, rs = reference(x, r, w, 1e-6)
        if residual:
            assert torch.equal(h, h_ref)
        assert_y(y, exact)
        assert ((rstd.double() - rs).abs() <= rs * U * 1.01).all()
        # the gradients
        dy = torch.randn((T, H), generator=gen, device=DEV).to(dtype)
        dh = torch.randn((T, H), generator=gen, device=DEV).to(dtype) if pad != 5 else None
        dx, dw = torch.full_like(y, 99.0), torch.full_like(w, 99.0)
        B.moe_rms_norm_backward(dy, x if h is None else h, w, rstd, dx, dw, B.rms_norm_scratch(T, H, x).fill_(0xff), dh=dh)
        z, d = h_ref.double() * rs[:, None], dy.double()
        g = d * w.double()
        more = dh.double() if dh is not None else torch.zeros_like(d)
        rs = rs[:, None]
        size, mean_abs = z.abs(), (g * z).abs().mean(1, keepdim=True)
        want = rs * (g - z * (g * z).mean(1, keepdim=True)) + more
        bound = half_step(want, dtype) + U * (
            8 * (rs * g.abs() + rs * size * mean_abs) + 48 * rs * size * mean_abs + want.abs() + more.abs())
        assert ((dx.double() - want).abs() <= bound).all()
        want = (d * z).sum(0)
        bound = half_step(want, w_dtype) + 100 * U * (d * z).abs().sum(0)
        assert ((dw.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T,H", [(1, 128), (5, 384), (64, 4096), (7, 7168), (3, 1024), (66, 256), (2, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_mxfp8_form_is_the_quantization_of_y(T, H, dtype):
    gen = torch.Generator(DEV).manual_seed(T + H)
    x, r = wide(gen, T, H, dtype, 0, 2.0), wide(gen, T, H, dtype, 16)
    x[T // 2, :64] = 0
    r[T // 2, :64] = 0                                      # two blocks of zeros
    w = (1.0 + 0.3 * torch.randn((H,), generator=gen, device=DEV)).to(dtype)
    y, h = torch.empty((T, H), dtype=dtype, device=DEV), torch.empty((T, H), dtype=dtype, device=DEV)
    codes = torch.full((T, H), 7, dtype=torch.uint8, device=DEV)
    scales = B.mx_scales_empty((T, H), DEV).fill_(7)
    B.moe_rms_norm(x, w, y, 1e-5, residual=r, h=h, codes=codes, scales=scales)
    h_ref, exact, _ = reference(x, r, w, 1e-5)
    assert torch.equal(h, h_ref)
    assert_y(y, exact)
    # the codes, from the format's definition on y
    b = y.double().view(T, -1, 32)
    top = b.abs().amax(2)
    e = (torch.frexp(top)[1] - 9).clamp(-127, 127)
    e = torch.where(top == 0, -127, e)
    want = torch.ldexp(b, -e[..., None].double()).clamp(-448, 448).float().to(torch.float8_e4m3fn)
    assert torch.equal(codes, want.view(T, H).view(torch.uint8))
    words = scales.view(H // 128, -1, 4)
    assert torch.equal(words[:, :T].permute(1, 0, 2).reshape(T, -1), (e + 127).to(torch.uint8))
    assert (words[:, T:] == 7).all()                        # padding words are not written
    if dtype == BF16:
        c2, s2 = torch.empty_like(codes), torch.full_like(scales, 7)
        B.moe_mx_quantize(y, c2, s2)
        assert torch.equal(codes, c2) and torch.equal(scales, s2)
    # without y
    c2, s2 = torch.empty_like(codes), torch.full_like(scales, 7)
    B.moe_rms_norm(x, w, None, 1e-5, residual=r, codes=c2, scales=s2)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("H", [96, 2048])
def test_memory_in_place(H):
    gen = torch.Generator(DEV).manual_seed(H)
    x, r, w = wide(gen, 50, H, BF16, 0), wide(gen, 50, H, BF16, 0), torch.ones((H,), device=DEV)
    y, h = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty((50,), device=DEV)
    B.moe_rms_norm(x, w, y, residual=r, h=h, rstd=rstd)
    for a, b in (("x", "r"), ("r", "x")):                   # h over one operand, y over the other
        t = {"x": x.clone(), "r": r.clone()}
        B.moe_rms_norm(t["x"], w, t[b], residual=t["r"], h=t[a])
        assert torch.equal(t[a], h) and torch.equal(t[b], y)
    t = x.clone()
    B.moe_rms_norm(t, w, t)
    B.moe_rms_norm(x, w, y)
    assert torch.equal(t, y)
    dy, dh = torch.randn_like(x), torch.randn_like(x)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = B.rms_norm_scratch(50, H, x)
    B.moe_rms_norm_backward(dy, h, w, rstd, dx, dw, ws, dh=dh)
    for name in ("dy", "dh"):
        t = {"dy": dy.clone(), "dh": dh.clone()}
        B.moe_rms_norm_backward(t["dy"], h, w, rstd, t[name], dw, ws, dh=t["dh"])
        assert torch.equal(t[name], dx)


def test_values_at_the_ends():
    H = 256
    w = torch.ones((H,), device=DEV)
    x = torch.zeros((6, H), dtype=BF16, device=DEV)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e-20                                            # squares far below eps
    x[4] = 1e15
    x[5, 0] = -0.0
    y = torch.empty_like(x)
    rstd = torch.empty((6,), device=DEV)
    B.moe_rms_norm(x, w, y, 1e-6, rstd=rstd)
    assert (y[0] == 0).all() and rstd[0].item() == pytest.approx(1e3, rel=1e-6)
    assert rstd[1] == 0 and torch.isnan(y[1, 3]) and (y[1, :3] == 0).all()     # as x / infinity
    assert torch.isnan(y[2]).all()
    assert torch.equal(y[3:5], rounded(reference(x, None, w, 1e-6)[1], BF16)[3:5])
    assert torch.signbit(y[5, 0]) and not torch.signbit(y[5, 1])
    # a product that leaves fp16
    x16 = torch.ones((1, H), dtype=F16, device=DEV)
    w16 = torch.full((H,), 65504.0, device=DEV)
    w16[1], w16[2] = 65519.9, 1e6
    y16 = torch.empty_like(x16)
    B.moe_rms_norm(x16, w16, y16, 1e-30)
    assert y16[0, 0] == 65504 and y16[0, 1] == 65504 and torch.isinf(y16[0, 2])


def test_other_rows_do_not_matter_and_bits_repeat():
    gen = torch.Generator(DEV).manual_seed(3)
    x, w = wide(gen, 700, 384, F16, 0), torch.ones((384,), device=DEV)
    y, y1 = torch.empty_like(x), torch.empty_like(x[:1])
    rstd = torch.empty((700,), device=DEV)
    B.moe_rms_norm(x, w, y, rstd=rstd)
    B.moe_rms_norm(x[137:138], w, y1)
    assert torch.equal(y[137:138], y1)
    dy = torch.randn_like(x)
    got = []
    for _ in range(2):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        B.moe_rms_norm_backward(dy, x, w, rstd, dx, dw, B.rms_norm_scratch(700, 384, x), dh=None)
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_operands_beyond_32_bits():
    T, H = 140_000, 16384                                   # 2.3e9 elements
    gen = torch.Generator(DEV).manual_seed(6)
    x = torch.zeros((T, H), dtype=BF16, device=DEV)
    x[-3:] = torch.randn((3, H), generator=gen, device=DEV)
    w = (1 + 0.1 * torch.randn((H,), generator=gen, device=DEV))
    y, rstd = torch.full_like(x, 99.0), torch.empty((T,), device=DEV)
    codes, scales = torch.empty((T, H), dtype=torch.uint8, device=DEV), B.mx_scales_empty((T, H), DEV)
    B.moe_rms_norm(x, w, y, rstd=rstd, codes=codes, scales=scales)
    assert (y[:-3] == 0).all()
    assert_y(y[-3:], reference(x[-3:], None, w, 1e-6)[1])
    c, s = torch.empty((3, H), dtype=torch.uint8, device=DEV), B.mx_scales_empty((3, H), DEV)
    B.moe_mx_quantize(y[-3:], c, s)
    assert torch.equal(codes[-3:], c) and torch.equal(scales[:, -3:], s.view(H // 128, 4, 4)[:, :3])
    dx, dw = torch.full_like(x, 99.0), torch.empty_like(w)
    B.moe_rms_norm_backward(y, x, w, rstd, dx, dw, B.rms_norm_scratch(T, H, x))
    dx3, dw3 = torch.empty_like(x[-3:]), torch.empty_like(w)
    B.moe_rms_norm_backward(y[-3:], x[-3:], w, rstd[-3:], dx3, dw3, B.rms_norm_scratch(3, H, x))
    assert (dx[:-3] == 0).all() and torch.equal(dx[-3:], dx3)
    assert ((dw - dw3).abs() <= 1e-5 * dw3.abs() + 1e-6).all()      # the same three terms, added in other places


def test_a_product_whose_factors_leave_fp32():
    x = torch.full((2, 64), 3e18, device=DEV)
    w = torch.full((64,), 1e25, device=DEV)                 # x w is beyond fp32, x rstd w is 1e25
    for t in (torch.float32, BF16):
        y = torch.empty((2, 64), dtype=t, device=DEV)
        B.moe_rms_norm(x.to(t), w, y)
        assert_y(y, reference(x.to(t), None, w, 1e-6)[1])


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=BF16, device=DEV), torch.ones((64,), device=DEV)
    B.moe_rms_norm(x, w, torch.empty_like(x))
    dw = torch.full_like(w, 99.0)
    B.moe_rms_norm_backward(x, x, w, torch.empty((0,), device=DEV), torch.empty_like(x), dw, B.rms_norm_scratch(0, 64, x))
    assert (dw == 0).all()


def test_gradient_against_differences():
    gen = torch.Generator(DEV).manual_seed(9)
    T, H, step = 3, 40, 2.0 ** -10
    x, w = torch.randn((T, H), generator=gen, device=DEV), 1 + 0.2 * torch.randn((H,), generator=gen, device=DEV)
    dy = torch.randn((T, H), generator=gen, device=DEV)
    rstd, y = torch.empty((T,), device=DEV), torch.empty_like(x)
    B.moe_rms_norm(x, w, y, 1e-6, rstd=rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    B.moe_rms_norm_backward(dy, x, w, rstd, dx, dw, B.rms_norm_scratch(T, H, x))

    def loss(x, w):
        out = torch.empty_like(x)
        B.moe_rms_norm(x, w, out, 1e-6)
        return (out.double() * dy.double()).sum().item()
    # central differences: their error is step^2 / 6 times a third derivative of order one, and the
    # outputs' rounding, sqrt(T H) 2^-24 / step at most: some 2^-14 / 2 of values of order one
    for t, c in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros_like(x)
        e[t, c] = step
        assert (loss(x + e, w) - loss(x - e, w)) / (2 * step) == pytest.approx(dx[t, c].item(), abs=2e-3)
    e = torch.zeros_like(w)
    e[7] = step
    assert (loss(x, w + e) - loss(x, w - e)) / (2 * step) == pytest.approx(dw[7].item(), abs=2e-3)


def test_captured_and_on_another_stream():
    gen = torch.Generator(DEV).manual_seed(4)
    T, H = 130, 2048
    x, r, w = wide(gen, T, H, BF16, 0), wide(gen, T, H, BF16, 0), torch.ones((H,), device=DEV)
    dy = torch.randn((T, H), device=DEV).to(BF16)
    bufs = dict(y=torch.empty_like(x), h=torch.empty_like(x), rstd=torch.empty((T,), device=DEV),
                codes=torch.empty((T, H), dtype=torch.uint8, device=DEV), scales=B.mx_scales_empty((T, H), DEV))
    dx, dw, ws = torch.empty_like(x), torch.empty_like(w), B.rms_norm_scratch(T, H, x)

    def step():
        B.moe_rms_norm(x, w, bufs["y"], residual=r, h=bufs["h"], rstd=bufs["rstd"], codes=bufs["codes"],
                       scales=bufs["scales"])
        B.moe_rms_norm_backward(dy, bufs["h"], w, bufs["rstd"], dx, dw, ws)
    step()
    want = {k: v.clone() for k, v in bufs.items()} | {"dx": dx.clone(), "dw": dw.clone()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
    x0 = x.clone()
    x.copy_(r)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(bufs["y"], want["y"])
    x.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    got = bufs | {"dx": dx, "dw": dw}
    for k, v in want.items():
        if k == "scales":
            assert torch.equal(got[k].view(H // 128, -1, 4)[:, :T], v.view(H // 128, -1, 4)[:, :T])
        else:
            assert torch.equal(got[k], v), k
