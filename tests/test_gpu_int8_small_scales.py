"""int8 codes of rows whose scale is close to fp32's smallest normal number, where the remainder of a quotient has no
fp32 number of its own: still the codes of IEEE division, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import int8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows_of_ties(low, high, n, seed):
    """Rows of scales from 2^low to 2^high (some full, some with few fraction bits) that hold, besides 127 scales, every
    tie (2 m + 1) / 2 scales and its neighbours at one and two ulps."""
    g = np.random.default_rng(seed)
    scale = np.ldexp(1 + g.random(n), g.integers(low, high, n)).astype(np.float32)
    few = np.arange(n) % 3 == 0
    scale[few] = (scale[few].view(np.uint32) & np.uint32(0xfff00000)).view(np.float32)
    amax = (scale.astype(np.float64) * 127).astype(np.float32)
    s = np.maximum(amax / np.float32(127), np.float32(2.0 ** -126))
    mid = (s.astype(np.float64)[:, None] * (np.arange(-127, 127) + 0.5)).astype(np.float32)
    parts = [amax[:, None], np.zeros((n, 1), np.float32)]
    for to in (-np.inf, np.inf):
        one = np.nextafter(mid, np.float32(to))
        parts += [one, np.nextafter(one, np.float32(to))]
    x = np.concatenate(parts + [mid], 1)
    x = np.clip(x, -amax[:, None], amax[:, None])
    return np.concatenate([x, np.zeros((n, -x.shape[1] % 8), np.float32)], 1)


@pytest.mark.parametrize("low,high", [(-126, -125), (-126, -110), (-110, -95), (-102, -98)])
def test_quantiser_divides_as_ieee_does_down_to_the_smallest_scale(low, high):
    from split_weight_expert_amd import api
    x = rows_of_ties(low, high, 400, -low)
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    s = torch.empty(len(x), device=DEV)
    api.quantize_tokens_int8(torch.from_numpy(x).to(DEV), q, s)
    want, ws = o8.rows(x)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), want)


def test_rows_below_the_smallest_scale():
    """amax / 127 under 2^-126: the scale is 2^-126 and the codes are those of the subnormal values."""
    from split_weight_expert_amd import api
    g = np.random.default_rng(3)
    x = np.ldexp(g.integers(-(1 << 20), 1 << 20, (60, 136)).astype(np.float64), -g.integers(129, 149, (60, 1))).astype(np.float32)
    x[:, :64] = np.ldexp(np.arange(64) - 31.5, -126).astype(np.float32) * (np.arange(60) % 2)[:, None]
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    s = torch.empty(len(x), device=DEV)
    api.quantize_tokens_int8(torch.from_numpy(x).to(DEV), q, s)
    want, ws = o8.rows(x)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_half_of_the_largest(dt):
    """A value of exactly half of its row's largest is 63.5 steps in real arithmetic; its code is that of the quotient by
    the scale as it is stored, amax / 127 rounded: 63 or 64, as IEEE division says."""
    from split_weight_expert_amd import api
    amax = torch.linspace(1, 2, 1000).to(dt).float()
    x = torch.zeros(1000, 16)
    x[:, 0], x[:, 1], x[:, 2] = amax, amax / 2, -amax / 2
    x = x.to(dt)
    q = torch.empty(1000, 16, dtype=torch.int8, device=DEV)
    s = torch.empty(1000, device=DEV)
    api.quantize_tokens_int8(x.to(DEV), q, s)
    want, ws = o8.rows(x.float().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), want)
    assert set(np.unique(want[:, 1])) == {63, 64}


@pytest.mark.parametrize("T,H", [(300, 136), (40, 1000), (9, 7168), (3, 40000)])
@pytest.mark.parametrize("exponent", [-126, -121, -112])
def test_norms_divide_as_ieee_does(T, H, exponent):
    """The norm's codes are those of its fp32 output, whose scale a small weight brings down."""
    from split_weight_expert_amd import api
    g = torch.Generator().manual_seed(H)
    # whole numbers over few values: many quotients at and beside ties
    x = torch.randint(-254, 255, (T, H), generator=g).float()
    x[:, 0] = 254
    w = torch.full((H,), 2.0 ** exponent)
    y, q, s = torch.empty(T, H, device=DEV), torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    api.branch_add_rmsnorm(x.to(DEV), None, None, w.to(DEV), 1e-6, y=y, q=q, q_scale=s)
    want, ws = o8.rows(y.cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), want)
