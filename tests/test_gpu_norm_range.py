"""The norm's rounding at the ends of fp32's range: rows near the largest number, elements far below
their row under large weights, products that leave the range. y is the exact value rounded once (fp32:
within 2^-24 (1 + 2^-20), half a step and what 48 bits leave out) for every finite row,
of 16-bit rows where an element's h rstd is at least 2^-190 and the result no bf16 below its normal numbers."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from norm_reference import U, assert_y, reference, rounded

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def norm(x, w, eps=1e-6, **kw):
    y = torch.empty_like(x)
    B.moe_rms_norm(x, w, y, eps, **kw)
    return y


@pytest.mark.parametrize("dtype,tops", [(F32, (1e13, 1e15, 1e19, 1e30, 1e37, 1e38, 3e38)), (BF16, (1e13, 1e15, 1e19, 1e37, 1e38, 3e38))])
@pytest.mark.parametrize("H", [33, 256, 1003, 4096, 16384])
def test_rows_of_large_numbers(dtype, tops, H):
    gen = torch.Generator(DEV).manual_seed(H)
    w = 1 + 0.3 * torch.randn((H,), generator=gen, device=DEV)
    for top in tops:
        x = ((2 * torch.rand((40, H), generator=gen, device=DEV) - 1) * top).to(dtype)
        rstd = torch.empty((40,), device=DEV)
        y = norm(x, w, rstd=rstd)
        exact, rs = reference(x, w, 1e-6)
        assert_y(y, exact)
        # rstd is rounded twice at most, to steps of 2^-149 below fp32's normal numbers
        assert ((rstd.double() - rs).abs() <= rs * U * 1.01 + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_small_elements_under_large_weights(dtype):
    """h rstd far below fp32's normal numbers (16-bit values: down to 2^-190), where the weight brings y back."""
    H = 256
    gen = torch.Generator(DEV).manual_seed(1)
    x = torch.randn((60, H), generator=gen, device=DEV)
    x = torch.sign(x) * x.abs().clamp(min=2.0 ** -6)
    # rows' rms is 2^63 at most, beside elements of 2^-116 at least: h rstd from 2^-179 on
    x *= torch.exp2(torch.randint(-110, 60, (60, H), generator=gen, device=DEV).double()).float()
    x[:, 0] = 1e20
    x[::2, 1:40] = 1e-20
    x[::3, 40:60] = 1e-27
    x[1::3, 60:70] = 0.0
    x = x.to(dtype)
    for scale in (1e10, 1e20, 1e30, 1e38):
        w = torch.randn((H,), generator=gen, device=DEV).clamp(-3, 3) * scale
        w[5::7] = 0.0
        y, exact = norm(x, w), reference(x, w, 1e-6)[0]
        normal = exact.abs() >= 2.0 ** -126
        assert_y(y[normal], exact[normal])
        assert ((y.double() - exact).abs()[~normal] <= 2.0 ** -134 + 2.0 ** -149).all()
        assert (y[exact == 0] == 0).all()


def test_small_results():
    """Weights that take y to the smallest numbers and below: a bf16 value below its normal numbers is within
    half its step and a step of fp32's, the others are rounded once."""
    H = 256
    gen = torch.Generator(DEV).manual_seed(4)
    x32 = torch.randn((300, H), generator=gen, device=DEV)
    for scale in (1e-30, 1e-37, 1e-39):
        w = torch.randn((H,), generator=gen, device=DEV) * scale
        assert_y(norm(x32, w), reference(x32, w, 1e-6)[0])
        x = x32.to(BF16)
        y, exact = norm(x, w), reference(x, w, 1e-6)[0]
        normal = exact.abs() >= 2.0 ** -126
        assert_y(y[normal], exact[normal])
        assert ((y.double() - exact).abs()[~normal] <= 2.0 ** -134 + 2.0 ** -149).all()
    x = x32.to(F16)
    for scale in (1e-4, 1e-6, 1e-8):
        w = torch.randn((H,), generator=gen, device=DEV) * scale
        assert_y(norm(x, w), reference(x, w, 1e-6)[0])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_products_beyond_the_range_beside_others(dtype):
    """A product beyond the type, or an infinite weight, gives infinity whatever its neighbours are."""
    H = 512
    gen = torch.Generator(DEV).manual_seed(2)
    x = torch.randn((300, H), generator=gen, device=DEV)
    x += torch.sign(x) * 0.5                                # no element near 0
    x = x.to(dtype)
    w = 1 + 0.3 * torch.randn((H,), generator=gen, device=DEV)
    w[3::16], w[9::16] = 3.4e38, float("inf")
    x[:, 3::16] *= 100                                      # z of 3 and more: z w leaves fp32
    y, plain = norm(x, w), w.clone()
    plain[3::16], plain[9::16] = 1.0, 1.0
    exact = reference(x, plain, 1e-6)[0]
    ends = torch.zeros((H,), dtype=torch.bool, device=DEV)
    ends[3::16], ends[9::16] = True, True
    assert_y(y[:, ~ends], exact[:, ~ends])
    assert torch.isinf(y[:, ends]).all()
    assert torch.equal(torch.signbit(y[:, ends]), torch.signbit(x[:, ends]))


def test_products_at_the_largest_number():
    """Products around fp32's largest number: rounded as 64 bits say, infinity from the border on."""
    H = 256
    gen = torch.Generator(DEV).manual_seed(3)
    x = torch.randn((200, H), generator=gen, device=DEV)
    x[:, ::2] = 1.0
    for dtype in (F32, BF16):
        h = x.to(dtype)
        rs = reference(h, torch.ones((H,), device=DEV), 1e-6)[1].mean()
        w = (3.4028235e38 / rs * (1 + 2.0 ** -18 * torch.randn((H,), generator=gen, device=DEV).double())).clamp(max=3.4028234e38).float()
        y, exact = norm(h, w), reference(h, w, 1e-6)[0]
        want = rounded(exact, dtype)
        if dtype == F32:
            # the border of infinity is FLT_MAX (1 + 2^-25): within 2^-44 of it either is right
            sure = (exact.abs() / (3.4028234663852886e38 * (1 + 2.0 ** -25)) - 1).abs() > 2.0 ** -44
            assert torch.equal(torch.isinf(y)[sure], torch.isinf(want)[sure])
            fin = torch.isfinite(want) & torch.isfinite(y)
            assert_y(y[fin], exact[fin])
        else:
            assert torch.equal(y, want)
