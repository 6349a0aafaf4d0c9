"""Rows of the largest widths, 2^31 - 1 elements (the boundary: 2^31 - 8): the last column's successor passes 31 bits."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_layer import DEV

pytestmark = pytest.mark.gpu

UB16 = 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def spots(H):
    """Columns that are not zero: the first, the last, and some on both sides of 2^30 and of the last 2048."""
    return [0, 7, 2047, 2048, (1 << 30) - 1, 1 << 30, H - 2056, H - 2048, H - 2047, H - 9, H - 8, H - 1]


def check(H, z, out, y, w, eps):
    at = torch.tensor(spots(H), device=DEV)
    # powers of two: the squares and their sum are exact in fp32; the mean, the root, two products and y's rounding
    if out is not None:
        assert torch.equal(out[0, at].float(), z) and int(torch.count_nonzero(out)) == len(at)
    if y is not None:
        v = z.double()
        n = v / ((v * v).sum() / H + eps).sqrt() * w
        assert ((y[0, at].double() - n).abs() <= (UB16 + 8 * 2.0 ** -24) * n.abs()).all()
        assert int(torch.count_nonzero(y)) == len(at)


def row(H):
    x = torch.zeros(1, H, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor(spots(H), device=DEV)
    z = torch.exp2(torch.arange(len(at), device=DEV) % 4).float()
    x[0, at] = z.to(torch.bfloat16)
    return x, z


@pytest.mark.parametrize("H", [(1 << 31) - 1, (1 << 31) - 8])
def test_add_rmsnorm_of_the_widest_row(H):
    from split_weight_expert_amd import api
    x, z = row(H)
    w = torch.full((H,), 1.5, dtype=torch.bfloat16, device=DEV)
    so, y = torch.full_like(x, 7), torch.full_like(x, 7)
    api.add_rmsnorm(x, None, w, 1e-6, so, y)
    torch.cuda.synchronize()
    check(H, z, so, y, 1.5, 1e-6)


def test_combine_add_rmsnorm_of_the_widest_row():
    from split_weight_expert_amd import api
    H = (1 << 31) - 8
    x, z = row(H)
    so = torch.full_like(x, 7)
    api.combine_add_rmsnorm(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, 1, device=DEV), 0, None, None, 0.0,
                            sum_out=so)
    torch.cuda.synchronize()
    check(H, z, so, None, None, 0.0)


@pytest.mark.parametrize("dt,H", [("f32", 33000), ("f32", 1 << 20), ("f32", (1 << 25) + 3), ("f32", (1 << 30) + 8), ("bf16", (1 << 31) - 8)])
def test_a_wide_row_of_equal_elements(dt, H):
    """Terms that are all alike round all the same way once the sum is far larger than each: the mean square of a row
    of 1.09375 (its square is exact) is off by the roundings of 7 additions in a vector, of the sum to fp32, of 8
    additions in the workgroup, of H and of the division, half of which (9 u) are on the root; the root, its reciprocal
    and the product with z add 3 u, and the output its rounding."""
    from split_weight_expert_amd import api
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dt]
    x = torch.full((1, H), 1.09375, dtype=t, device=DEV)
    w = torch.ones(H, dtype=t, device=DEV)
    y = torch.empty_like(x)
    api.add_rmsnorm(x, None, w, 0.0, y=y)
    torch.cuda.synchronize()
    u = 2.0 ** -24
    low, high = float(y.min()), float(y.max())
    tol = 12 * u + (UB16 if dt == "bf16" else u)
    assert 1 - tol <= low and high <= 1 + tol, (low, high)


def test_a_wide_boundary_of_equal_elements():
    from split_weight_expert_amd import api
    H = 1 << 24
    x = torch.full((3, H), 0.546875, device=DEV)
    inv = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    y = torch.empty(1, H, device=DEV)
    api.combine_add_rmsnorm(x, inv, torch.full((1, 2), 0.5, device=DEV), 1, None, torch.ones(H, device=DEV), 0.0, y=y)
    torch.cuda.synchronize()
    assert float((y.double() - 1).abs().max()) <= 13 * 2.0 ** -24
