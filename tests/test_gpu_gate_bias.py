"""Group-limited gates whose balance biases are large and of both signs, against fp64.

A bias of +B on some experts and -B on others lets the sum of a group's two best choices cancel: it is of a
score's size, but carries the rounding of numbers of B's size.  The choice must still be the fp64 one.
"""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_layer import DEV, check_gate, gen, make_gate, run_gate, torch_gate

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def biases(E, groups, B, g):
    """One expert of each group lifted and the others pushed down; signs at random; and sizes from 1 to B at random."""
    one = torch.full((groups, E // groups), -B, device=DEV)
    one[:, 0] = B
    sign = torch.where(torch.rand(E, generator=g, device=DEV) < 0.5, B, -B)
    size = torch.sign(sign) * torch.exp(torch.rand(E, generator=g, device=DEV) * torch.log(torch.tensor(B, device=DEV)))
    return one.reshape(E), sign, size


# E, groups, kept, group_top, k, T: 16 lanes of 4, 8 and 16 experts a token, 64 lanes, and more groups than lanes
SHAPES = [(4, 2, 1, 2, 2, 1_000_000), (16, 8, 4, 2, 4, 400_000), (60, 12, 5, 2, 6, 50_000), (128, 8, 4, 2, 8, 50_000),
          (256, 8, 4, 2, 8, 100_000), (256, 8, 4, 2, 8, 2000), (256, 8, 4, 1, 8, 20_000), (255, 5, 2, 2, 9, 20_000),
          (512, 8, 4, 2, 8, 20_000), (1024, 16, 4, 2, 8, 10_000), (160, 80, 20, 2, 8, 4000)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [1e2, 1e3, 1e4, 1e5])
@pytest.mark.parametrize("E,groups,kept,top,k,T", SHAPES)
def test_groups_of_large_biases_of_both_signs(E, groups, kept, top, k, T, B, score):
    g = gen(E + T + int(B))
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
    gate = make_gate(k, score, groups, kept, top, True, 2.5)
    for n, balance in enumerate(biases(E, groups, B, g)):
        idx, _ = run_gate(logits, gate, balance)
        oi, _ = torch_gate(logits, gate, balance)
        assert torch.equal(idx, oi), (n, int((idx != oi).any(1).sum()))


@pytest.mark.parametrize("T", [1, 64, 4000])
def test_a_cancelling_pair(T):
    """Two groups whose sums are 1.38905 and 1.38938; in fp32, where 10^4 has a spacing of 2^-10, the other way round."""
    logits = torch.tensor([[1.5034595, 0.28578004, 1.7111572, 0.16997097]], device=DEV).repeat(T, 1)
    balance = torch.tensor([1e4, -1e4, 1e4, -1e4], device=DEV)
    gate = make_gate(2, "sigmoid", 2, 1, 2)
    idx, w = run_gate(logits, gate, balance)
    assert (idx == torch.tensor([2, 3], device=DEV)).all()
    check_gate(logits[:1], gate, balance, idx[:1], w[:1])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,kept,top,k,T", [(64, 8, 3, 2, 6, 64), (256, 8, 3, 2, 6, 64), (256, 8, 3, 1, 6, 2100), (512, 8, 3, 2, 6, 64)])
def test_infinite_and_overflowing_biases(E, groups, kept, top, k, T, score):
    """An expert pinned by +inf, and groups whose sum of two biases passes the largest fp32 number."""
    g = gen(E + T)
    gs = E // groups
    logits = torch.randn(T, E, generator=g, device=DEV)
    pinned = torch.randn(E, generator=g, device=DEV) * 0.05
    pinned[[3, gs + 1, 4 * gs, 4 * gs + 1, 6 * gs]] = float("inf")
    huge = torch.randn(E, generator=g, device=DEV) * 0.05
    for i, v in ((1, 3e38), (2, 3.2e38), (5, -3e38)):
        huge[i * gs:(i + 1) * gs] = v
    huge[7 * gs:] = -3.3e38
    low = torch.full((E,), -3e38, device=DEV)
    low[: 2 * gs] = -float("inf")                       # groups of no live expert come behind the lowest sums
    for balance in (pinned, huge, low, -huge):
        gate = make_gate(k, score, groups, kept, top, True, 1.5)
        idx, w = run_gate(logits, gate, balance)
        check_gate(logits, gate, balance, idx, w)
