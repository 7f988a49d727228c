"""The norm's gradients where a block goes through several rows: rows fetched ahead, sums that alternate,
dweight added over a block's rows, blocks that are a row short, and the second launch's rounds.

The bounds are those of the formulas' roundings, each at most 2^-24 of a magnitude. dx takes four to z and
g, two to the bracket, one to the stream's gradient, and the mean of the row at most 4 (vectors) x 8 + 10
(the threads) additions in a row and three roundings of each product. dweight takes three roundings of
each product and in a row at most 64 additions of a thread's rows, 8 of a block's warps, and 10 + 8 + 6 of the
second launch (ten parts, rounds of 640 parts, the threads of a column). Half a step of the type is added
for the last rounding."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from norm_reference import U, half_step, reference, rounded, wide

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def check(h, w, rstd64, dy, dh, dx, dw):
    rs = rstd64[:, None]
    for a in range(0, h.shape[0], 4096):                    # 64 bits of some rows at a time
        s = slice(a, a + 4096)
        z, d = h[s].double() * rs[s], dy[s].double()
        g = d * w.double()
        more = dh[s].double() if dh is not None else torch.zeros_like(d)
        mean, mean_abs = (g * z).mean(1, keepdim=True), (g * z).abs().mean(1, keepdim=True)
        want = rs[s] * (g - z * mean) + more
        bound = half_step(want, dx.dtype) + U * (
            8 * (rs[s] * g.abs() + rs[s] * z.abs() * mean_abs) + 48 * rs[s] * z.abs() * mean_abs + want.abs() + more.abs())
        assert ((dx[s].double() - want).abs() <= bound).all()
        one, size = (d * z).sum(0), (d * z).abs().sum(0)
        total, magnitude = (one, size) if a == 0 else (total + one, magnitude + size)
    assert ((dw.double() - total).abs() <= half_step(total, dw.dtype) + 100 * U * magnitude).all()


# rows of a warp (three of them and more), of a block, single elements; some blocks a row short
SIZES = [(20000, 128), (20001, 384), (20000, 512), (9000, 24), (3001, 1003), (20003, 200), (3000, 33), (3001, 2048),
         (3000, 4096), (1999, 7168), (1501, 16384), (1500, 16376), (901, 16383), (2000, 8191)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F32), (F16, F16), (F32, F32)])
def test_gradients_of_several_rows_a_block(T, H, dtype, w_dtype):
    gen = torch.Generator(DEV).manual_seed(T + H)
    for pad, stream in ((0, True), (0, False), (5, True)):  # pad 5: h's rows at odd places
        h = wide(gen, T, H, dtype, pad, 3.0)
        w = (1.0 + 0.3 * torch.randn((H,), generator=gen, device=DEV)).to(w_dtype)
        dy = wide(gen, T, H, dtype, 0)
        dh = wide(gen, T, H, dtype, 0) if stream else None
        rs = reference(h, w, 1e-6)[1]
        dx, dw = torch.full((T, H), 99.0, dtype=dtype, device=DEV), torch.full_like(w, 99.0)
        ws = B.rms_norm_scratch(T, H, h).fill_(0xff)
        B.moe_rms_norm_backward(dy, h, w, rs.float(), dx, dw, ws, dh=dh)
        check(h, w, rs, dy, dh, dx, dw)
        # the gradient in the place of dy or dh
        for name in ("dy", "dh") if stream and pad == 0 else ():
            t = {"dy": dy.clone(), "dh": dh.clone()}
            dw2 = torch.full_like(w, 99.0)
            B.moe_rms_norm_backward(t["dy"], h, w, rs.float(), t[name], dw2, ws.fill_(0xff), dh=t["dh"])
            assert torch.equal(t[name], dx) and torch.equal(dw2, dw)


def test_the_most_rows_of_a_thread():
    """64 rows a block and more: blocks beyond a wave, parts of dweight over several rounds."""
    T, H = 64 * 2000 + 17, 1032
    gen = torch.Generator(DEV).manual_seed(5)
    h, dy = wide(gen, T, H, BF16, 0), wide(gen, T, H, BF16, 0)
    dy.add_(0.25)                                           # terms of one sign: what is lost or doubled shows
    h.abs_()
    w = torch.ones((H,), device=DEV)
    rs = reference(h, w, 1e-6)[1]
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    B.moe_rms_norm_backward(dy, h, w, rs.float(), dx, dw, B.rms_norm_scratch(T, H, h).fill_(0xff))
    check(h, w, rs, dy, None, dx, dw)


def test_forward_of_many_rows():
    gen = torch.Generator(DEV).manual_seed(6)
    for T, H, dtype in ((5001, 1003, F16), (3001, 2048, BF16), (9001, 128, BF16)):
        x, r = wide(gen, T, H, dtype, 3), wide(gen, T, H, dtype, 0)
        w = 1.0 + 0.3 * torch.randn((H,), generator=gen, device=DEV)
        y, h = torch.empty((T, H), dtype=dtype, device=DEV), torch.empty((T, H), dtype=dtype, device=DEV)
        B.moe_rms_norm(x, w, y, residual=r, h=h)
        assert torch.equal(h, rounded(x.double() + r.double(), dtype))
        assert torch.equal(y, rounded(reference(h, w, 1e-6)[0], dtype))
