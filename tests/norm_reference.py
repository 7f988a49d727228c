"""The norm's formulas in 64 bits, and its values rounded once."""
import torch

F32 = torch.float32
U = 2.0 ** -24


def rounded(v, dtype):
    """Finite 64-bit values rounded once to `dtype` (a conversion would round twice, by way of fp32)."""
    f = v.float()
    if dtype == F32:
        return f
    low = v - f.double()
    bits = f.view(torch.int32)
    odd = torch.where((bits & 1 == 0) & (low != 0), torch.sign(low * torch.sign(f.double())).int(), 0)
    return (bits + odd).view(F32).to(dtype)


def wide(gen, T, H, dtype, pad, scale=1.0):
    return torch.randn((T, H + pad), generator=gen, device="cuda").mul_(scale).to(dtype)[:, :H]


def reference(h, weight, eps):
    """y and rstd of the stream h."""
    h64 = h.double()
    rstd = 1.0 / torch.sqrt(h64.square().mean(1, keepdim=True) + eps)
    return h64 * rstd * weight.double(), rstd[:, 0]


def half_step(v, dtype):
    return torch.finfo(dtype).eps / 2 * v.abs().clamp(min=torch.finfo(dtype).smallest_normal)


def assert_y(y, exact):
    """Equal to the exact value rounded once; fp32, from a value good to some 48 bits, within 2^-24 (1 + 2^-20), and
    infinity where the exact value rounds to it."""
    want = rounded(exact, y.dtype)
    if y.dtype == F32:
        over = torch.isinf(want)
        assert torch.equal(y[over], want[over])
        assert ((y.double() - exact).abs() <= exact.abs() * U * (1 + 2.0 ** -20) + 2.0 ** -149)[~over].all()
    else:
        assert torch.equal(y, want)
