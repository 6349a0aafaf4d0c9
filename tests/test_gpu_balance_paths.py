"""The balance loss and the gate's gradient on the launches that test_gpu_balance.py leaves out: lane layouts of long batches,
thousands of sequences (each workgroup searches its own), and the z loss of tokens without live logits.  Tolerances: there."""
import numpy as np
import pytest
import torch

from oracle import balance as ob
from tests.test_gpu_balance import DEV, U, api, check_gradient, check_loss, routed, run_loss, spread  # noqa: F401

pytestmark = pytest.mark.gpu


# more than 4096 tokens: 16 lanes for 33 to 64 experts, 32 for 257 to 512, 64 above, and for k > 16 as few tokens have
LONG = [(4500, 60, 6), (4200, 384, 8), (5000, 512, 16), (4099, 33, 1), (4100, 640, 4), (4200, 100, 20), (4097, 17, 17), (4200, 512, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", LONG)
def test_long_batches(api, T, E, k, renormalize, score):
    l, idx, g = routed(T, E, k, T + E)
    gate = api.Gate(k=k, score=score, renormalize=renormalize, scale=1.5)
    offsets = [3, 1000, 1000, T - 7]
    o, off, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, offsets)
    check_loss(o, S, l, idx, score, offsets)
    check_gradient(api, l, idx, gate, offsets, g, o["counts"][:S], off)


# a workgroup asks for every sequence's start up to 2048 sequences (loss) or 1022 (gradient) and searches beyond
@pytest.mark.parametrize("T,S", [(1500, 1022), (1500, 1023), (3000, 2048), (3000, 2049), (5003, 3000), (300, 5000), (70, 4097)])
def test_thousands_of_sequences(api, T, S):
    """Sequences of random lengths, many of them empty, tokens before the first and behind the last."""
    E, k = 24, 3
    l, idx, g = routed(T, E, k, S)
    offsets = sorted(torch.randint(T // 50 + 1, T - T // 40, (S + 1,), generator=g).tolist())
    gate = api.Gate(k=k, score="sigmoid")
    o, off, _ = run_loss(api, l.to(DEV), idx.to(DEV), gate, offsets)
    check_loss(o, S, l, idx, "sigmoid", offsets)
    check_gradient(api, l, idx, gate, offsets, g, o["counts"][:S], off)


def test_most_sequences(api):
    """2^20 sequences, one token in each of some: every other one is empty and has zeros."""
    T, E, k, S = 1000, 8, 2, 1 << 20
    l, idx, g = routed(T, E, k, 9)
    at = sorted(torch.randperm(S, generator=g)[:T].tolist())          # the sequence of each token
    lengths = np.zeros(S, np.int64)
    lengths[at] = 1
    offsets = np.concatenate([[0], lengths.cumsum()]).tolist()
    o, _, _ = run_loss(api, l.to(DEV), idx.to(DEV), api.Gate(k=k), offsets)
    counts, probs, balance, z = ob.losses(l.numpy(), idx.numpy(), "softmax", list(range(T + 1)))
    rel = (2.2 * spread(l.numpy()) + 12) * 2 * U + 552 * U
    live = torch.tensor(at, device=DEV)
    got = {n: t[live].double().cpu().numpy() for n, t in o.items()}
    assert (got["counts"] == counts).all() and (np.abs(got["probs"] - probs) <= rel * probs + 1e-36).all()
    assert (np.abs(got["balance"] - balance) <= (rel + 64 * U) * balance + 1e-36).all()
    for t in o.values():
        rest = t[:S].clone()
        rest[live] = 0
        assert (rest == 0).all() and (t[S:] == -7).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_z_loss_of_dead_logits(api, score):
    """A sequence of each token: NaN and -inf take no part in its logsumexp, a token of none other has 0, the lowest fp32
    value is a logit like any other; and one sequence of all of them."""
    l, idx, _ = routed(9, 20, 4, 5)
    l[3, 5] = float("nan")
    l[4, :19] = float("-inf")
    l[5] = float("-inf")
    l[6] = float("nan")
    l[7, 2] = torch.finfo(torch.float32).min
    gate = api.Gate(k=4, score=score)
    live = l.nan_to_num(nan=0.0, neginf=0.0).clamp(min=-100).numpy()
    f = np.abs(live).max(1) + np.log(20.0)              # |logsumexp| at most
    for offsets in (list(range(10)), [0, 9]):
        o, _, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, offsets)
        z = ob.losses(l.numpy(), idx.numpy(), score, offsets)[3]
        # logits that count for more than 2^-24 lie within 17 of the largest
        rel = (2.2 * 17 + 12) * 2 * U
        b = f if S == 9 else np.array([f.max()])
        assert (np.abs(o["z"][:S].double().cpu().numpy() - z) <= 2 * b * (4 * U * b + rel) + 16 * U * z).all()
        if S == 9:
            assert (o["z"][5:7] == 0).all() and o["z"][4].item() > 0 and z[4] == pytest.approx(float(l[4, 19]) ** 2)
