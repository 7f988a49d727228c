"""Sums so long that one tile works on them for more than a second."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def test_a_group_of_many_rows():
    """dw of 4e8 rows in one group, all zeros but some: 6.2e6 k-blocks of 64 rows on one pair of SMs. The
    sums are whole numbers, exact in any order."""
    R, N, K = 400_000_033, 8, 8
    a, b = torch.zeros((R, N), dtype=BF16, device=DEV), torch.zeros((R, K), dtype=BF16, device=DEV)
    rows = torch.tensor([0, 1, 63, 64, 123_456_789, 200_000_000, R - 65, R - 2, R - 1], device=DEV)
    gen = torch.Generator(DEV).manual_seed(1)
    a[rows] = torch.randint(-3, 4, (len(rows), N), generator=gen, device=DEV).to(BF16)
    b[rows] = torch.randint(-3, 4, (len(rows), K), generator=gen, device=DEV).to(BF16)
    dw, ws = torch.full((2, N, K), 77.0, dtype=BF16, device=DEV), B.grouped_workspace(2)
    B.moe_grouped_wgrad(a, b, torch.tensor([0, R, R], dtype=torch.int32, device=DEV), dw, ws)
    assert B.moe_get_device_error(ws) == 0
    assert torch.equal(dw[0], (a[rows].float().t() @ b[rows].float()).to(BF16)) and (dw[1] == 0).all()


def test_a_long_reduction():
    """out of 4e8 columns of x: the same through a matrix [K, N]."""
    R, K, N = 20, 400_000_008, 8
    x, w = torch.zeros((R, K), dtype=BF16, device=DEV), torch.zeros((1, K, N), dtype=BF16, device=DEV)
    cols = torch.tensor([0, 1, 63, 64, 123_456_789, 200_000_000, K - 65, K - 2, K - 1], device=DEV)
    gen = torch.Generator(DEV).manual_seed(2)
    x[:, cols] = torch.randint(-3, 4, (R, len(cols)), generator=gen, device=DEV).to(BF16)
    w[0, cols] = torch.randint(-3, 4, (len(cols), N), generator=gen, device=DEV).to(BF16)
    out, ws = torch.full((R, N), 77.0, dtype=BF16, device=DEV), B.grouped_workspace(1)
    B.moe_grouped_mm(x, w, torch.tensor([0, R], dtype=torch.int32, device=DEV), out, ws, transposed=True)
    assert B.moe_get_device_error(ws) == 0
    assert torch.equal(out, (x[:, cols].float() @ w[0, cols].float()).to(BF16))
