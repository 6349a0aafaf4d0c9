"""The gate over a sliced router product, at sizes where each token layout and the sorted keys are taken."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_layer import (DEV, assert_tail, check_gate, gate_outputs, gen, make_gate, route_inputs, route_ws, run_gate,
                                  torch_gate)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# T, H, E, k, groups, kept, group_top: ragged last waves; sorted keys above 8192 tokens of up to 256 experts and above 2048 of
# up to 1024, each with many rounds and with few
CASES = [(9001, 2048, 256, 8, 8, 4, 2), (8193, 7168, 256, 8, 8, 4, 2), (9001, 2048, 200, 6, 1, 1, 1), (9002, 2048, 256, 2, 8, 4, 1),
         (2305, 2048, 1024, 8, 16, 4, 2), (2306, 4096, 1000, 12, 1, 1, 1), (2305, 2048, 1024, 3, 16, 4, 1),
         (4097, 2048, 128, 8, 8, 4, 2), (1777, 2048, 60, 6, 12, 5, 2), (515, 2048, 320, 8, 8, 3, 2), (77, 7168, 250, 8, 5, 2, 2)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,H,E,k,groups,kept,top", CASES)
def test_route_gate_of_sliced_products(T, H, E, k, groups, kept, top, score):
    from split_weight_expert_amd import api
    x, wr, bias = route_inputs(T, H, E, "bf16", T + E)
    # slices are there to be added: a plan of one needs no workspace
    assert api.route_gate_workspace_bytes(T, H, E, api.BF16) >= 2 * T * E * 4
    x[T - 1, 0] = float("nan")                          # the last token of a ragged wave has no live expert
    balance = torch.randn(E, generator=gen(E), device=DEV) * 0.05
    balance[E // 3] = -float("inf")
    want = (x.cpu().double() @ wr.cpu().double().t()).to(DEV)
    for b, bb in ((None, balance), (bias, balance), (bias, None)):
        buf, ws = route_ws(T, H, E, x)
        gate = make_gate(k, score, groups, kept, top, True, 2.5)
        idx, w, lo = gate_outputs(T, k, E)
        api.route_gate(x, wr, gate, lo[:T], idx[:T], w[:T], ws, bias=b, balance_bias=bb)
        torch.cuda.synchronize()
        assert_tail(T, idx, w, lo)
        assert (buf[:256] == 0xAB).all() and (buf[len(buf) - 256:] == 0xAB).all(), "wrote outside the workspace"
        n = T - 1
        assert torch.equal(lo[:n].double(), want[:n] if b is None else want[:n] + b.double())
        assert lo[n].isnan().all() and (idx[n] == -1).all() and (w[n] == 0).all()
        oi, _ = torch_gate(lo[:n], gate, bb)
        assert torch.equal(idx[:n], oi), int((idx[:n] != oi).any(1).sum())
        few = slice(n - 70, n)
        check_gate(lo[few], gate, bb, idx[few], w[few])
        # the gate alone, on these logits, gives the same bits
        i2, w2 = run_gate(lo[:T], gate, bb)
        assert torch.equal(i2, idx[:T]) and torch.equal(w2.view(torch.int32), w[:T].view(torch.int32))
