"""int8 experts at the limits that the call promises: sums that fp32 cannot hold, K of 65536 in either product, A's rows wider
than the quantiser's registers; and how many of A's codes differ from those of fp64's.  Tolerances: test_gpu_int8.py."""
import numpy as np
import pytest
import torch

from oracle import int8 as o8
from tests.test_gpu_int8 import DEV, Layer, U, api  # noqa: F401

pytestmark = pytest.mark.gpu


def reload(L):
    for e, (b, s) in enumerate([(0, e) if e < L.G // 2 else (1, e - L.G // 2) for e in range(L.G)]):
        L.store.load_int8(b, s, L.w13[e].to(DEV), L.s13[e].to(DEV), L.w2[e].to(DEV), L.s2[e].to(DEV))


def cancelling(w, rng, every):
    """Large weights of one sign in the first half of K, their negatives in the second, but for one in `every` columns,
    which is one step off: against equal halves the sum grows past 2^24 and comes back to a small odd or even number."""
    n, K = w.shape
    first = rng.integers(100, 127, (n, K // 2))
    off = np.where(rng.random((n, K // 2)) < 1.0 / every, rng.integers(0, 2, (n, K // 2)) * 2 - 1, 0)
    return torch.from_numpy(np.concatenate([first, off - first], 1).astype(np.int8))


@pytest.mark.parametrize("rows,H,I", [([40, 7], 8192, 128), ([130, 20], 8192, 256)])
def test_sums_that_pass_2_24_and_come_back(api, rows, H, I):
    """GEMM1: 4096 products near 113 * 113 are 5e7, beyond fp32's whole numbers, and the sum is some hundreds."""
    rng = np.random.default_rng(1)
    L = Layer(api, rows, H, I, 1)
    for e in range(L.G):
        L.w13[e] = cancelling(L.w13[e], rng, 64)
    half = rng.integers(100, 128, (L.T, H // 2)).astype(np.int8)
    q = np.concatenate([half, half], 1)
    sums = q.astype(np.int64) @ L.w13[0].numpy().astype(np.int64).T
    steps = np.cumsum(q[0].astype(np.int64) * L.w13[0][0].numpy())
    assert np.abs(steps).max() > 1 << 25 and np.abs(sums).max() < 1 << 15 and (sums % 2 == 1).any()
    L.q.copy_(torch.from_numpy(q))
    L.qs.fill_(0.01)
    L.s13 = 0.05 + 0.1 * torch.rand(L.s13.shape, generator=torch.Generator().manual_seed(2))
    reload(L)
    L.check()


def test_second_sums_that_pass_2_24_and_come_back(api):
    """GEMM2: A's two halves are equal, every channel's weights cancel but for a few."""
    H, I, rng = 256, 8192, np.random.default_rng(3)
    L = Layer(api, [30, 5], H, I, 4)
    L.q.copy_(torch.randint(60, 128, L.q.shape, generator=torch.Generator().manual_seed(5), dtype=torch.int8))
    L.qs.fill_(0.01)
    for e in range(L.G):
        w = torch.randint(110, 128, (I // 2, H), generator=torch.Generator().manual_seed(e), dtype=torch.int8)
        L.w13[e] = torch.cat([w, w, w, w])                # gate and up rows, both halves of I alike, all of one sign
        L.w2[e] = cancelling(L.w2[e], rng, 64)
    L.s13.fill_(1e-4)
    reload(L)
    L.check()
    a = L.a()[0].astype(np.int64)
    assert (a[:, :I // 2] == a[:, I // 2:]).all() and a.min() > 60
    steps = np.cumsum(a[0] * L.w2[0][0].numpy())
    assert np.abs(steps).max() > 1 << 24 and abs(steps[-1]) < 1 << 15


@pytest.mark.parametrize("rows,H,I", [([3, 2], 65536, 128), ([5, 0, 2], 256, 65536), ([4], 512, 32896), ([70], 256, 33024)])
def test_widest_products(api, rows, H, I):
    """K = 65536 in GEMM1 and in GEMM2; A's rows above 32768 columns, which the quantiser reads twice."""
    Layer(api, rows, H, I, H + I).check()


def test_largest_sum_of_all(api):
    """65536 products of -128 and -128 are 2^30; every A is the same, and so is every code."""
    L = Layer(api, [3], 65536, 128, 5, T=3, extreme=True)
    L.s13.fill_(2.0 ** -28)
    reload(L)
    L.qs.copy_(torch.tensor([1.0, 0.5, 2.0]))
    L.run(1)
    a, s = L.a()
    x = L.qs.double().cpu().numpy()[L.src.numpy()] * 2.0 ** 30 * 2.0 ** -28
    A = x / (1 + np.exp(-x)) * x
    assert (a == 127).all()
    assert (np.abs(s - A / 127) <= A / 127 * ((3.5 * x + 12) * 2 * U + 4 * U)).all()


def test_few_codes_of_a_move(api):
    """A code differs from fp64's where A / scale is closer to a tie than its error, at most 127 steps of A's error and twice
    the scale's: of values spread over a step, twice that distance's share, and twice it again for chance."""
    L = Layer(api, [300, 0, 40, 200], 1024, 1024, 17)
    moved = L.check()
    q, qs = L.q.cpu().numpy(), L.qs.cpu().numpy()
    most = max(np.abs(o8.gate_up(q, qs, L.w13[e].numpy(), L.s13[e].numpy())[1]).max() for e in (0, 2, 3))
    rel = (3.5 * most + 12) * 2 * U
    assert moved / 3 <= 2 * 2 * 127 * (2 * rel + 4 * U)
