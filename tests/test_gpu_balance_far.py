"""The sigmoid gate's gradient and losses where logits are far from 0: still to a few roundings.

Bounds in units of 2^-24, every operation at most half an ulp (1) and the hardware's exponential, reciprocal and logarithm an
ulp (2): e^l has 3.  A lone sigmoid's s (1 - s): e^l 3 on each side of it at most (6), 1 + e once in each of two factors (2),
the reciprocal twice (4), three products (3), and scale and d_w's product one more: 16, taken as 17 for their products.
A softmax share of n like terms: e^l 3, or for logits up to 8, where the rounded exponent l log2 e is used as it is, 2 and that
exponent's half ulp (6) and the constant's (2): 10; the sum's 10 and its additions (8 in a lane, 5 of 32 lanes), the reciprocal 2,
the product 1: 36; logsumexp 3 and what the sum's 23 are of a number of 4 or more: 6; d_z / N 2 and two products 2: 49, taken
as 52."""
import numpy as np
import pytest
import torch

from oracle import balance as ob

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.mark.parametrize("T,E,k", [(64, 16, 4), (200, 256, 8), (5000, 60, 6)])
def test_slope_of_a_lone_sigmoid(T, E, k):
    """Logits from -80 to 80: the gradient of weights that are not renormalised, which nothing else adds to."""
    from split_weight_expert_amd import api
    g = torch.Generator().manual_seed(T)
    l = (torch.rand(T, E, generator=g) * 2 - 1) * 80
    idx = torch.rand(T, E, generator=g).topk(k, 1).indices.int()
    dw = torch.randn(T, k, generator=g)
    out = torch.empty(T, E, device=DEV)
    api.gate_backward(l.to(DEV), idx.to(DEV), api.Gate(k=k, score="sigmoid", renormalize=False, scale=1.5), out, dw.to(DEV))
    want, size = ob.backward(l.numpy(), idx.numpy(), "sigmoid", False, 1.5, None, dw.double().numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= 17 * U * size + 1e-37).all()


@pytest.mark.parametrize("at", [2.0, 6.9, 8.0, 30.0, 62.0, 77.0])
@pytest.mark.parametrize("T,E", [(300, 32), (200, 256), (6000, 256)])
def test_shares_of_large_logits(T, E, at):
    """Logits within 1 of a large one: the z loss's gradient, whose parts are a softmax's shares."""
    from split_weight_expert_amd import api
    g = torch.Generator().manual_seed(T + E)
    l = at + torch.rand(T, E, generator=g) * 2 - 1
    out = torch.empty(T, E, device=DEV)
    api.gate_backward(l.to(DEV), torch.zeros(T, 2, dtype=torch.int32, device=DEV), api.Gate(k=2, score="sigmoid"), out,
                      d_z=torch.ones(1, device=DEV))
    want, _ = ob.backward(l.numpy(), np.zeros((T, 2), np.int32), "sigmoid", True, 1.0, None, None, None, np.ones(1))
    assert (np.abs(out.double().cpu().numpy() - want) <= 52 * U * np.abs(want)).all()
