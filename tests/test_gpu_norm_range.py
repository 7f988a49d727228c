"""The norm's rounding at the ends of fp32's range: products that leave it. y is the exact value rounded
once (fp32: within 2^-24 (1 + 2^-20), half a step and what 48 bits leave out)."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B
from norm_reference import assert_y, reference, rounded

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
