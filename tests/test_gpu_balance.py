"""The balance loss, the z loss, per-expert counts and the gate's gradient on the GPU against the fp64 oracle.

Tolerances.  e^x is 2^(x log2 e): the product's rounding is an absolute error of |x| 1.5 2^-24 in the exponent, so with x
down to -D its relative error is at most (1.1 D + 2) 2^-23; a probability takes two of them (its own and its sum's, or a
sigmoid's), and eight more roundings: rel = (2.2 D + 12) 2^-23.  Means add the roundings of their sums, at most 512 terms
in a row and 40 of trees: 552 2^-24.  Terms below 2^-120 may be flushed: an absolute 1e-36."""
import numpy as np
import pytest
import torch

from oracle import balance as ob

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_weight_expert_amd import api
    return api


def spread(l):
    """Largest distance of a logit that matters from its token's largest, and of a sigmoid's from 0."""
    l = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(invalid="ignore", all="ignore"):
        top = np.nanmax(l, 1, keepdims=True)
        d = np.nanmax(np.abs(top - l))
        return float(min(max(np.nan_to_num(d), min(np.nan_to_num(np.nanmax(np.abs(l))), 40.0)), 110.0))


def routed(T, E, k, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * scale + torch.randn(E, generator=g) * 0.5
    return l, l.topk(k, 1).indices.to(torch.int32), g


def run_loss(api, l, idx, gate, offsets=None, stream=None, ws=None):
    T, E = l.shape
    S = 1 if offsets is None else len(offsets) - 1
    o = dict(counts=torch.full((S + 1, E), -7, dtype=torch.int32, device=DEV), probs=torch.full((S + 1, E), -7.0, device=DEV),
             balance=torch.full((S + 1,), -7.0, device=DEV), z=torch.full((S + 1,), -7.0, device=DEV))
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if ws is None:
        ws = torch.full((api.balance_loss_workspace_bytes(T, E, S),), 0xff, dtype=torch.uint8, device=DEV)
    api.balance_loss(l, idx, gate, **{n: t[:S] for n, t in o.items()}, ws=ws, seq_offsets=off, stream=stream)
    return o, off, S


def check_loss(o, S, l, idx, score, offsets):
    for t in o.values():
        assert (t[S:] == -7).all(), "written behind the last sequence"
    counts, probs, balance, z = ob.losses(l.cpu().numpy(), idx.cpu().numpy(), score, offsets)
    rel = (2.2 * spread(l.cpu().numpy()) + 12) * 2 * U + 552 * U
    np.testing.assert_array_equal(o["counts"][:S].cpu().numpy(), counts)
    got = {n: t[:S].double().cpu().numpy() for n, t in o.items()}
    assert (np.abs(got["probs"] - probs) <= rel * probs + 1e-36).all()
    assert (np.abs(got["balance"] - balance) <= (rel + 64 * U) * balance + 1e-36).all()
    # logsumexp = top + log(sum): an ulp of each, the sum's relative error; squared, that twice |lse| times
    f = np.where(np.isfinite(l.cpu().numpy()), np.abs(l.cpu().numpy()), 0).max() + np.log(l.shape[1])
    assert (np.abs(got["z"] - z) <= 2 * f * (4 * U * f + rel) + (552 + 8) * U * z).all()


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (64, 16, 4), (65, 17, 3), (100, 32, 8), (333, 33, 6), (64, 64, 8), (1000, 60, 6),
          (257, 128, 8), (512, 129, 8), (4096, 256, 8), (4097, 256, 8), (77, 257, 32), (300, 512, 12), (130, 1000, 32),
          (64, 1024, 8), (20000, 24, 4)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_losses(api, T, E, k, score):
    l, idx, _ = routed(T, E, k, T + E)
    o, _, S = run_loss(api, l.to(DEV), idx.to(DEV), api.Gate(k=k, score=score))
    check_loss(o, S, l, idx, score, None)


OFFSETS = [(100, [0, 100]), (100, [0, 0, 100]), (100, [0, 1, 2, 2, 99, 100]), (100, [5, 37, 90]), (1000, [0, 0, 0, 0]),
           (1000, [999, 1000, 1000]), (5000, list(range(0, 5001, 50))), (3000, [0, 7, 2049, 2050, 2999])]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,offsets", OFFSETS)
def test_sequences(api, T, offsets, score):
    E, k = 96, 6
    l, idx, g = routed(T, E, k, T)
    idx[::7, 1] = -1
    idx[::11, 2] = E
    gate = api.Gate(k=k, score=score, scale=1.5)
    o, off, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, offsets)
    check_loss(o, S, l, idx, score, offsets)
    check_gradient(api, l, idx, gate, offsets, g, o["counts"][:S], off)


def check_gradient(api, l, idx, gate, offsets, g, counts, off, parts="wbz"):
    T, E = l.shape
    S = 1 if offsets is None else len(offsets) - 1
    dw = torch.randn(T, gate.k, generator=g) if "w" in parts else None
    db = torch.randn(S, generator=g) * T if "b" in parts else None
    dz = torch.randn(S, generator=g) if "z" in parts else None
    out = torch.full((T + 1, E), -7.0, device=DEV)

    def dev(t):
        return None if t is None else t.to(DEV)
    api.gate_backward(l.to(DEV), idx.to(DEV), gate, out[:T], dev(dw), counts if db is not None else None, dev(db), dev(dz), off)
    assert (out[T:] == -7).all()
    n = [None if t is None else t.double().numpy() for t in (dw, db, dz)]
    d, size = ob.backward(l.numpy(), idx.numpy(), gate.score, gate.renormalize, gate.scale, offsets, *n)
    got = out[:T].double().cpu().numpy()
    # every term is a product of at most two probabilities (or a slope), a mean factor and sums over E or k of them
    rel = 2 * (2.2 * spread(l.numpy()) + 12) * 2 * U + (64 + gate.k) * U
    assert (np.abs(got - d) <= rel * size + 1e-36).all(), np.max(np.abs(got - d) / (size + 1e-30))
    return got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient(api, T, E, k, score, renormalize):
    l, idx, g = routed(T, E, k, 3 * T + E)
    gate = api.Gate(k=k, score=score, renormalize=renormalize, scale=2.5)
    counts = torch.from_numpy(ob.losses(l.numpy(), idx.numpy(), score)[0]).to(DEV)
    check_gradient(api, l, idx, gate, None, g, counts, None)


@pytest.mark.parametrize("parts", ["w", "b", "z", "wb", "wz", "bz"])
def test_gradients_of_some_parts(api, parts):
    for score in ("softmax", "sigmoid"):
        l, idx, g = routed(200, 40, 5, 8)
        counts = torch.from_numpy(ob.losses(l.numpy(), idx.numpy(), score)[0]).to(DEV)
        check_gradient(api, l, idx, api.Gate(k=5, score=score), None, g, counts, None, parts)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_same_expert_twice_and_dropped_slots(api, score):
    l, idx, g = routed(50, 12, 4, 21)
    idx[:, 1] = idx[:, 0]
    idx[::3, 2] = -1
    idx[::5] = -1                             # tokens without an expert
    idx[::4, 3] = 12
    for renormalize in (True, False):
        gate = api.Gate(k=4, score=score, renormalize=renormalize)
        o, off, S = run_loss(api, l.to(DEV), idx.to(DEV), gate)
        check_loss(o, S, l, idx, score, None)
        got = check_gradient(api, l, idx, gate, None, g, o["counts"][:S], off, "w")
        assert (got[::5] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_dead_logits(api, score):
    """Logits of NaN and -inf take no part; tokens of none other add nothing; the lowest fp32 value is a logit."""
    l, idx, g = routed(40, 20, 4, 5)
    l[3, 5] = float("nan")
    l[4, :19] = float("-inf")
    l[5] = float("-inf")
    l[6] = float("nan")
    l[7, 2] = torch.finfo(torch.float32).min
    l[8] = torch.finfo(torch.float32).min
    idx[4] = torch.tensor([19, 3, 2, -1])
    gate = api.Gate(k=4, score=score)
    off = [0, 8, 9, 40]
    o, offd, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, off)
    counts, probs, balance, z = ob.losses(l.numpy(), idx.numpy(), score, off)
    rel = (2.2 * spread(l.numpy()) + 12) * 2 * U + 552 * U
    for s in (0, 2):                         # sequence 1's z overflows fp32
        assert np.allclose(o["z"][s].item(), z[s], rtol=4 * rel, atol=0) or s == 0
    assert np.isinf(o["z"][1].item())
    assert np.allclose(o["probs"][:S].cpu().numpy(), probs, rtol=rel, atol=1e-36)
    assert np.allclose(o["balance"][:S].cpu().numpy(), balance, rtol=2 * rel, atol=1e-36)
    dw, db = torch.randn(40, 4, generator=g), torch.randn(3, generator=g)
    out = torch.empty(40, 20, device=DEV)
    api.gate_backward(l.to(DEV), idx.to(DEV), gate, out, dw.to(DEV), o["counts"][:S], db.to(DEV), None, offd)
    d, size = ob.backward(l.numpy(), idx.numpy(), score, True, 1.0, off, dw.double().numpy(), db.double().numpy())
    got = out.double().cpu().numpy()
    assert (np.abs(got - d) <= (4 * rel + 70 * U) * size + 1e-36).all()
    assert (got[5] == 0).all() and (got[6] == 0).all() and got[3, 5] == 0 and (got[4, :19] == 0).all()


def test_infinite_logits(api):
    """Logits of +inf share the softmax; the z loss is infinite there and the other gradients stay finite."""
    l, idx, g = routed(9, 8, 2, 4)
    l[2, 1] = l[2, 6] = float("inf")
    idx[2] = torch.tensor([1, 6])
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            gate = api.Gate(k=2, score=score, renormalize=renormalize)
            o, off, S = run_loss(api, l.to(DEV), idx.to(DEV), gate)
            assert np.isinf(o["z"][0].item())
            probs = ob.losses(l.numpy(), idx.numpy(), score)[1]
            assert np.allclose(o["probs"][:1].cpu().numpy(), probs, rtol=1e-5)
            dw, db = torch.randn(9, 2, generator=g), torch.ones(1)
            out = torch.empty(9, 8, device=DEV)
            api.gate_backward(l.to(DEV), idx.to(DEV), gate, out, dw.to(DEV), o["counts"][:S], db.to(DEV))
            assert torch.isfinite(out).all()
            d, size = ob.backward(l.numpy(), idx.numpy(), score, renormalize, 1.0, None, dw.double().numpy(), db.double().numpy())
            assert (np.abs(out.double().cpu().numpy() - d) <= 1e-5 * size + 1e-36).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-500.0, -60.0, -29.9, -30.1, 60.0, 500.0])
def test_shifted_logits(api, score, shift):
    """Scores that underflow (or saturate) all together: probabilities and renormalised weights are those of the limit."""
    l, idx, g = routed(60, 24, 4, 6)
    l = l + shift
    gate = api.Gate(k=4, score=score)
    o, off, S = run_loss(api, l.to(DEV), idx.to(DEV), gate)
    check_loss(o, S, l, idx, score, None)
    # the logits are given in fp32, and so is the fp64 oracle's input: no error of the shift itself
    check_gradient(api, l, idx, gate, None, g, o["counts"][:S], off)


def test_gradient_against_differences_of_the_losses(api):
    """The GPU's gradient against central differences of the GPU's own losses and weights along random directions.  A loss
    of size L has an error of about 1e-6 L, a difference over 2h one of 1e-6 L / h; the third derivatives are below 10 L."""
    T, E, k = 512, 32, 4
    l, idx, g = routed(T, E, k, 12, scale=1.0)
    off = [0, 100, 512]
    w = torch.rand(T, k, generator=g, dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        gate = api.Gate(k=k, score=score, scale=1.5)

        def total(l):
            o, _, S = run_loss(api, l.float().to(DEV), idx.to(DEV), gate, off)
            tw = ob.weights(l.float().numpy(), idx.numpy(), score, True, 1.5)
            return o["balance"][0].item() * 3 - o["balance"][1].item() + 0.1 * o["z"][:S].sum().item() + (tw * w.numpy() / T).sum()
        o, offd, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, off)
        out = torch.empty(T, E, device=DEV)
        api.gate_backward(l.to(DEV), idx.to(DEV), gate, out, (w / T).float().to(DEV), o["counts"][:S],
                          torch.tensor([3.0, -1.0], device=DEV), torch.full((2,), 0.1, device=DEV), offd)
        h = 0.02
        for i in range(4):
            v = torch.randn(T, E, generator=g, dtype=torch.float64)
            if i == 3:
                v = out.double().cpu() / out.double().cpu().norm() * 20
            diff = (total(l.double() + h * v) - total(l.double() - h * v)) / (2 * h)
            L = 8.0
            assert abs(diff - (out.double().cpu() * v).sum().item()) <= 1e-6 * L / h + 10 * L * h * h / 6 + 1e-4


def test_repeats_its_bits_on_any_stream_in_any_workspace(api):
    l, idx, _ = routed(3000, 100, 6, 2)
    l, idx = l.to(DEV), idx.to(DEV)
    gate, off = api.Gate(k=6, score="sigmoid"), [0, 1000, 1001, 3000]
    a, _, _ = run_loss(api, l, idx, gate, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.zeros(api.balance_loss_workspace_bytes(100000, 100, 50), dtype=torch.uint8, device=DEV)
    b, _, _ = run_loss(api, l, idx, gate, off, ws=big)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c, _, _ = run_loss(api, l, idx, gate, off)
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])


def test_no_tokens(api):
    l, idx = torch.empty(0, 10, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    o, off, S = run_loss(api, l, idx, api.Gate(k=2), [0, 0, 0])
    assert all((t[:S] == 0).all() and (t[S:] == -7).all() for t in o.values())
    api.gate_backward(l, idx, api.Gate(k=2), torch.empty(0, 10, device=DEV), torch.empty(0, 2, device=DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_padding_of_any_content(api, score):
    """Rows before the first and behind the last sequence may hold anything: they change no loss, and get no gradient of one."""
    T, E, k = 90, 24, 3
    l, idx, g = routed(T, E, k, 31)
    off = [4, 30, 70]
    gate = api.Gate(k=k, score=score)
    a, offd, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, off)
    db, dz = torch.randn(2, generator=g).to(DEV), torch.randn(2, generator=g).to(DEV)
    want = torch.empty(T, E, device=DEV)
    api.gate_backward(l.to(DEV), idx.to(DEV), gate, want, None, a["counts"][:S], db, dz, offd)
    for n, v in enumerate((float("inf"), float("nan"), float("-inf"), torch.finfo(torch.float32).max)):
        l[n], l[70 + n], l[80, n] = v, v, v
        idx[n], idx[70 + n] = -(1 << 31) + n, (1 << 31) - 1 - n
    b, _, _ = run_loss(api, l.to(DEV), idx.to(DEV), gate, off)
    assert all(torch.equal(a[n], b[n]) for n in a)
    out = torch.empty(T, E, device=DEV)
    api.gate_backward(l.to(DEV), idx.to(DEV), gate, out, None, b["counts"][:S], db, dz, offd)
    assert torch.equal(out, want) and (out[:4] == 0).all() and (out[70:] == 0).all()


def test_two_calls_at_once(api):
    """Calls on two streams, each with a workspace of its own, enqueued without waiting for one another."""
    gate = api.Gate(k=4, score="sigmoid")
    sets = []
    for i in range(2):
        l, idx, _ = routed(6000 + i, 200, 4, i)
        sets.append((l.to(DEV), idx.to(DEV)))
    want = [run_loss(api, *s, gate)[0] for s in sets]
    ws = [torch.empty(api.balance_loss_workspace_bytes(6001, 200, 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run_loss(api, *sets[i], gate, ws=ws[i])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], want[i][n]) for i in range(2) for o in got[i] for n in o)


def test_a_long_batch(api):
    """Chunks of 4096 tokens: 2^20 + 3 tokens in two sequences, against sums in fp64."""
    T, E, k = (1 << 20) + 3, 8, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    l = torch.randn(T, E, device=DEV, generator=g)
    idx = l.topk(k, 1).indices.int()
    o, _, S = run_loss(api, l, idx, api.Gate(k=k), [0, 5, T])
    p = torch.softmax(l.double(), 1)
    for s, (a, b) in enumerate(((0, 5), (5, T))):
        assert torch.equal(o["counts"][s].long(), torch.bincount(idx[a:b].reshape(-1).long(), minlength=E))
        # D is below 12: (2.2 * 12 + 12) 2^-23 and the sums' 552 2^-24
        assert torch.allclose(o["probs"][s].double(), p[a:b].mean(0), rtol=(2.2 * 12 + 12) * 2 * U + 552 * U, atol=0)


def test_offsets_out_of_range_stay_in_bounds(api):
    """Offsets below 0 or past T are taken as 0 and T."""
    l, idx, g = routed(100, 16, 2, 1)
    gate = api.Gate(k=2)
    o, _, S = run_loss(api, l.to(DEV), idx.to(DEV), gate, [-5, 40, 1 << 30])
    check_loss(o, S, l, idx, "softmax", [0, 40, 100])


def test_binding_refuses_wrong_tensors_on_the_gpu(api):
    T, E, S = 6, 8, 2
    gate = api.Gate(k=2)
    l, i = torch.zeros(T, E, device=DEV), torch.zeros(T, 2, dtype=torch.int32, device=DEV)
    good = dict(counts=torch.zeros(S, E, dtype=torch.int32, device=DEV), probs=torch.zeros(S, E, device=DEV),
                balance=torch.zeros(S, device=DEV), z=torch.zeros(S, device=DEV),
                ws=torch.zeros(1 << 16, dtype=torch.uint8, device=DEV),
                seq_offsets=torch.zeros(S + 1, dtype=torch.int32, device=DEV))
    for n, bad in (("counts", good["counts"].long()), ("probs", good["probs"][:1]), ("balance", good["balance"][:1]),
                   ("z", good["z"].double()), ("seq_offsets", good["seq_offsets"][:2]), ("seq_offsets", good["seq_offsets"].long()),
                   ("counts", good["counts"].cpu())):
        with pytest.raises(ValueError, match=n):
            api.balance_loss(l, i, gate, **dict(good, **{n: bad}))
    with pytest.raises(ValueError, match="topk_idx"):
        api.balance_loss(l, i.long(), gate, **good)
    with pytest.raises(Exception, match="ws is NULL"):
        api.balance_loss(l, i, gate, **dict(good, ws=None))
    d = torch.zeros(T, E, device=DEV)
    g = dict(d_w=torch.zeros(T, 2, device=DEV), counts=good["counts"], d_balance=good["balance"], d_z=good["z"],
             seq_offsets=good["seq_offsets"])
    for n, bad in (("d_w", g["d_w"][:, :1]), ("d_balance", torch.zeros(3, device=DEV)), ("d_z", torch.zeros(1, device=DEV)),
                   ("seq_offsets", good["seq_offsets"][:2])):
        with pytest.raises(ValueError, match=n):
            api.gate_backward(l, i, gate, d, **dict(g, **{n: bad}))
