"""The gate, the norms and the layer boundary (include/dwdp_layer.h) on the GPU against fp64.

Chosen experts are compared as whole numbers with the oracle's choice on the same fp32 logits.  Tolerances
count roundings: half a step of a type is u = finfo(type).eps / 2 of the value, fp32's u is 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import codecs
from oracle import layer as ol
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

DEV = "cuda"
U32 = 2.0 ** -24
UB16 = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------------------------ gate

def gate_outputs(T, k, E=None):
    """Outputs with two rows behind the last, which no call may touch."""
    idx = torch.full((T + 2, k), -77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 2, k), -77.0, device=DEV)
    lo = None if E is None else torch.full((T + 2, E), -77.0, device=DEV)
    return idx, w, lo


def assert_tail(T, *bufs):
    for b in bufs:
        assert (b[T:].float() == -77).all(), "rows behind the last were written"


def weight_tolerance(logits, idx, w):
    """Relative error of a weight in fp32.  Its factor exp(l - shift): the difference is rounded (and scaled to a
    power of two) with relative error 2 u, |d| of it enters the exponent, so 2 |d| u; the exponential, the
    denominator's few roundings, the sum of up to 1024 non-negative scores in a tree of at most 16 + 6 levels, the
    division and the scale add less than 40 u."""
    l = np.nan_to_num(logits.astype(np.float64), nan=-1e30, posinf=0.0, neginf=-1e30)
    sel = np.take_along_axis(l, np.maximum(idx, 0).astype(np.int64), 1)
    d = np.abs(sel - l.max(1, keepdims=True)) + np.abs(sel)
    return (40 + 2 * d) * U32 * np.abs(w)


def check_gate(logits, gate, balance, idx, w):
    ln = logits.cpu().numpy()
    bn = None if balance is None else balance.cpu().numpy()
    oi, ow = ol.gate(ln, gate.k, gate.score, bn, gate.n_groups, gate.topk_groups, gate.group_top, gate.renormalize,
                     gate.scale)
    gi, gw = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(gi, oi)
    # 2^-126 below: fp32 weights under the smallest normal number may be flushed
    tol = weight_tolerance(ln, oi, ow) + 2.0 ** -126
    assert (np.abs(gw - ow) <= tol).all(), float((np.abs(gw - ow) / np.maximum(tol, 1e-300)).max())


def run_gate(logits, gate, balance=None):
    from split_weight_expert_amd import api
    T = logits.shape[0]
    idx, w, _ = gate_outputs(T, gate.k)
    api.gate_topk(logits, gate, idx[:T], w[:T], balance_bias=balance)
    torch.cuda.synchronize()
    assert_tail(T, idx, w)
    return idx[:T], w[:T]


def make_gate(k, score="softmax", groups=1, kept=1, top=1, renorm=True, scale=1.0):
    from split_weight_expert_amd import api
    return api.Gate(k=k, score=score, n_groups=groups, topk_groups=kept, group_top=top, renormalize=renorm, scale=scale)


# T, E, k, groups, kept, group_top
GATE_SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 8, 8, 1, 1, 1), (5, 2, 1, 2, 1, 2), (64, 256, 8, 8, 4, 2),
    (65, 256, 8, 8, 4, 1), (130, 60, 6, 1, 1, 1), (131, 60, 4, 4, 2, 2), (77, 7, 3, 1, 1, 1), (300, 160, 6, 8, 3, 1),
    (333, 300, 7, 5, 2, 2), (17, 1024, 32, 1, 1, 1), (19, 1024, 32, 16, 2, 2), (9, 1024, 1, 1024, 1, 2),
    (21, 1000, 12, 8, 8, 2), (33, 512, 16, 32, 3, 2), (40, 128, 32, 1, 1, 1), (41, 96, 9, 12, 5, 2), (1025, 16, 2, 4, 2, 1),
    (50, 257, 3, 1, 1, 1), (12, 999, 5, 9, 4, 2), (15, 64, 8, 64, 8, 2), (70, 320, 10, 20, 10, 1), (29, 896, 8, 7, 2, 2),
    (2049, 256, 8, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,groups,kept,top", GATE_SHAPES)
def test_gate_matches_the_oracle(T, E, k, groups, kept, top, score, biased):
    g = gen(T * 1000 + E)
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
    balance = torch.randn(E, generator=g, device=DEV) * 0.1 if biased else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        gate = make_gate(k, score, groups, kept, top, renorm, scale)
        idx, w = run_gate(logits, gate, balance)
        check_gate(logits, gate, balance, idx, w)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top", [(256, 1, 1, 1), (256, 8, 4, 2), (160, 8, 3, 1), (60, 1, 1, 1),
                                               (1000, 8, 2, 2), (512, 16, 4, 2)])
def test_equal_and_nearly_equal_choices(E, groups, kept, top, score):
    """Rows of equal logits, logits from few values, neighbours in the last bit, and choices that a bias brings
    within a few units of 2^-24 of each other: the order is the fp64 one, equals to the lower expert."""
    T, k = 96, 7
    g = gen(E + top)
    logits = torch.empty(T, E, device=DEV)
    logits[0:16] = 0.75
    logits[16:40] = torch.randint(0, 4, (24, E), generator=g, device=DEV).float() * 0.5
    ulp = torch.randint(0, 3, (24, E), generator=g, device=DEV).float() * 2.0 ** -23
    logits[40:64] = 1.0 + ulp
    logits[64:80] = torch.randn(16, E, generator=g, device=DEV) * 1e-6
    logits[80:88] = torch.where(torch.rand(8, E, generator=g, device=DEV) < 0.5, 0.0, -0.0)
    logits[88:] = 30.0 + torch.randn(8, E, generator=g, device=DEV)      # sigmoids that fp32 rounds to 1
    balances = [None, torch.zeros(E, device=DEV), torch.randint(0, 3, (E,), generator=g, device=DEV).float() * 2.0 ** -22]
    for balance in balances:
        gate = make_gate(k, score, groups, kept, top)
        idx, w = run_gate(logits, gate, balance)
        if score == "sigmoid" and balance is not None:
            # above 36 sigmoids are equal in fp64 or nearly; the oracle's and the kernel's exponentials may then round
            # to different neighbours, so those rows are compared by the choice they reach, to 4 fp64 steps
            check_gate(logits[:88], gate, balance, idx[:88], w[:88])
            c = 1 / (1 + np.exp(-logits[88:].double().cpu().numpy())) + balance.double().cpu().numpy()
            oi, _ = ol.gate(logits[88:].cpu().numpy(), k, score, balance.cpu().numpy(), groups, kept, top)
            gi = idx[88:].cpu().numpy()
            if groups == 1:
                np.testing.assert_allclose(np.take_along_axis(c, gi.astype(np.int64), 1),
                                           np.take_along_axis(c, oi.astype(np.int64), 1), rtol=0, atol=4 * 2.0 ** -53)
        else:
            check_gate(logits, gate, balance, idx, w)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups,kept,top", [(24, 1, 1, 1), (256, 8, 4, 2), (256, 8, 4, 1), (160, 8, 3, 2), (1024, 4, 2, 2),
                                               (257, 1, 1, 1)])
def test_masked_rows_and_non_finite_values(E, groups, kept, top, renorm, score):
    inf, nan = float("inf"), float("nan")
    T, k = 40, 6
    g = gen(E * 7 + top)
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits[0] = -inf                                             # nothing left
    logits[1] = nan
    logits[2] = -inf
    logits[2, E - 1] = 0.5                                       # one expert left
    logits[3, : E // 2] = nan
    logits[4, 3] = inf                                           # the whole softmax
    logits[5, [1, 5, E - 2]] = inf
    logits[6] = torch.finfo(torch.float32).min                   # a mask of the type's lowest value, everywhere
    logits[7, 2:] = torch.finfo(torch.float32).min               # ... and nearly everywhere
    logits[8] = torch.finfo(torch.float32).max
    logits[9] -= 2000.0                                          # sigmoids that underflow
    logits[10] = torch.where(torch.rand(E, generator=g, device=DEV) < 0.9, -inf, logits[10])
    logits[11, ::2] = -inf
    logits[12] *= 1e30
    logits[13] *= 1e-30
    drained = torch.zeros(E, device=DEV)
    drained[torch.rand(E, generator=g, device=DEV) < 0.3] = -inf
    wide = torch.randn(E, generator=g, device=DEV) * 0.1
    wide[0], wide[1], wide[2] = nan, inf, -inf
    for balance in (None, drained, wide, torch.full((E,), -inf, device=DEV)):
        rows = torch.arange(T, device=DEV)
        if balance is not None:
            # scores that all underflow, with a bias: equal in fp64, or not, by the exponential's last bit
            rows = rows[(rows != 13)]
        gate = make_gate(k, score, groups, kept, top, renorm)
        l = logits[rows].contiguous()
        idx, w = run_gate(l, gate, balance)
        check_gate(l, gate, balance, idx, w)


def test_gate_single_rows_and_no_rows():
    from split_weight_expert_amd import api
    gate = make_gate(8, "sigmoid", 8, 4, 2)
    logits = torch.randn(37, 256, generator=gen(3), device=DEV)
    balance = torch.randn(256, generator=gen(4), device=DEV) * 0.05
    idx, w = run_gate(logits, gate, balance)
    for t in range(37):                                   # a row by itself gives the same bits
        i1, w1 = run_gate(logits[t:t + 1].contiguous(), gate, balance)
        assert torch.equal(i1[0], idx[t]) and torch.equal(w1[0], w[t])
    api.gate_topk(logits[:0], gate, idx[:0], w[:0])


def test_gate_takes_unaligned_logits():
    """Logits whose rows start at odd 4-byte addresses."""
    for E in (256, 61):
        gate = make_gate(5, "sigmoid", 1, 1, 1)
        store = torch.randn(1 + 50 * E, generator=gen(E), device=DEV)
        l = store[1:].view(50, E)
        idx, w = run_gate(l, gate)
        check_gate(l, gate, None, idx, w)


# ------------------------------------------------------------------------------------------------ route

ROUTE_SHAPES = [  # T, H, E, k, groups, kept, dtype
    (1, 7168, 256, 8, 8, 4, "bf16"), (2, 64, 8, 2, 1, 1, "bf16"), (16, 128, 16, 4, 4, 2, "bf16"), (17, 192, 24, 3, 1, 1, "bf16"),
    (63, 7168, 256, 8, 8, 4, "bf16"), (64, 1984, 60, 6, 1, 1, "bf16"), (65, 1024, 160, 6, 8, 3, "bf16"),
    (255, 512, 300, 7, 5, 2, "bf16"), (257, 2048, 256, 8, 8, 4, "bf16"), (1000, 576, 1000, 12, 8, 3, "bf16"),
    (1777, 1984, 60, 6, 1, 1, "bf16"), (2500, 1024, 256, 8, 8, 4, "bf16"), (4099, 512, 1024, 32, 1, 1, "bf16"),
    (9000, 256, 128, 4, 1, 1, "bf16"), (33, 64, 1, 1, 1, 1, "bf16"), (129, 320, 511, 8, 1, 1, "bf16"),
    (1, 16, 8, 2, 1, 1, "f32"), (300, 512, 24, 4, 1, 1, "f32"), (77, 1040, 256, 8, 8, 4, "f32"),
]


def route_inputs(T, H, E, dt, seed):
    """Tokens and weights on a grid, so that the logits are exact in fp32 in any order of summation."""
    g = gen(seed)

    def grid(t, step):
        return (t.to(torch.bfloat16).float() / step).round() * step
    x = grid(torch.randn(T, H, generator=g, device=DEV).clamp_(-7, 7), 2.0 ** -5)
    w = grid(torch.randn(E, H, generator=g, device=DEV) * H ** -0.5, 2.0 ** -14)
    b = grid(torch.randn(E, generator=g, device=DEV) * 0.5, 2.0 ** -10)
    return x.to(DT[dt]), w.to(DT[dt]), b


def route_ws(T, H, E, x):
    from split_weight_expert_amd import api
    n = api.route_gate_workspace_bytes(T, H, E, api.dtype_code(x))
    # exactly the bytes named, between guards
    buf = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device=DEV)
    return buf, buf[256:256 + n] if n else None


@pytest.mark.parametrize("T,H,E,k,groups,kept,dt", ROUTE_SHAPES)
def test_route_gate_matches_the_oracle(T, H, E, k, groups, kept, dt):
    from split_weight_expert_amd import api
    x, wr, bias = route_inputs(T, H, E, dt, T + H + E)
    balance = torch.randn(E, generator=gen(E), device=DEV) * 0.05
    buf, ws = route_ws(T, H, E, x)
    ref = x.double().cpu() @ wr.double().cpu().t()
    for score, b, bb in (("sigmoid", None, balance), ("softmax", bias, None)):
        gate = make_gate(k, score, groups, kept, min(2, E // groups), True, 2.5)
        idx, w, lo = gate_outputs(T, k, E)
        api.route_gate(x, wr, gate, lo[:T], idx[:T], w[:T], ws, bias=b, balance_bias=bb)
        torch.cuda.synchronize()
        assert_tail(T, idx, w, lo)
        assert (buf[:256] == 0xAB).all() and (buf[len(buf) - 256:] == 0xAB).all(), "wrote outside the workspace"
        want = ref if b is None else ref + b.double().cpu()
        assert torch.equal(lo[:T].cpu().double(), want)
        check_gate(lo[:T], gate, bb, idx[:T], w[:T])


@pytest.mark.parametrize("T,H,E,k,groups,kept,dt", [
    (513, 1056, 256, 8, 8, 4, "f32"), (1030, 2080, 72, 6, 1, 1, "f32"), (700, 1040, 512, 8, 4, 2, "f32"), (70, 7168, 300, 7, 5, 2, "f32"),
    (9000, 64, 320, 4, 1, 1, "f32"), (2500, 416, 1000, 12, 8, 3, "f32"), (3000, 1024, 33, 4, 1, 1, "f32"), (80, 7168, 256, 8, 8, 4, "bf16"),
    (96, 7168, 256, 8, 8, 4, "bf16"), (40, 5376, 452, 12, 2, 2, "bf16"), (1000, 512, 128, 4, 1, 1, "bf16"), (2000, 64, 1000, 8, 1, 1, "bf16"),
    (3, 4096, 1024, 8, 16, 4, "bf16"), (1681, 2048, 168, 9, 8, 1, "bf16"),
    (9000, 32, 1000, 8, 1, 1, "f32"), (9000, 64, 1000, 8, 1, 1, "bf16"), (17000, 64, 300, 8, 1, 1, "bf16"), (12000, 64, 128, 4, 1, 1, "bf16"),
])
def test_route_gate_of_every_tile_and_slice(T, H, E, k, groups, kept, dt):
    """Small and large products of both types, in one slice and in several, with ragged tiles and K steps."""
    test_route_gate_matches_the_oracle(T, H, E, k, groups, kept, dt)


@pytest.mark.parametrize("T,H,E", [(7, 1008, 68), (200, 1024, 200), (600, 1056, 256), (300, 4096, 200), (1100, 1040, 100)])
def test_route_gate_random_fp32_values(T, H, E):
    """A logit's error is that of H rounded products and an fp32 sum of them in any order."""
    from split_weight_expert_amd import api
    g = gen(T)
    x = torch.randn(T, H, generator=g, device=DEV)
    wr = torch.randn(E, H, generator=g, device=DEV) * H ** -0.5
    gate = make_gate(6, "sigmoid")
    idx, w, lo = gate_outputs(T, 6, E)
    api.route_gate(x, wr, gate, lo[:T], idx[:T], w[:T], route_ws(T, H, E, x)[1])
    xd, wd = x.double(), wr.double()
    bound = (xd.abs() @ wd.abs().t().contiguous()) * (H + 1) * U32 * 1.01      # 1.01: the products of errors
    assert ((lo[:T].double() - xd @ wd.t().contiguous()).abs() <= bound).all()
    check_gate(lo[:T], gate, None, idx[:T], w[:T])


def test_route_gate_random_values():
    """Ordinary bf16 values: a logit's error is that of an fp32 sum of H exact products in any order."""
    from split_weight_expert_amd import api
    for T, H, E in ((5, 7168, 256), (200, 2048, 96), (3000, 1024, 256)):
        g = gen(T)
        x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
        wr = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).to(torch.bfloat16)
        gate = make_gate(6, "sigmoid")
        idx, w, lo = gate_outputs(T, 6, E)
        api.route_gate(x, wr, gate, lo[:T], idx[:T], w[:T], route_ws(T, H, E, x)[1])
        xd, wd = x.double(), wr.double()
        bound = (xd.abs() @ wd.abs().t().contiguous()) * H * U32
        assert ((lo[:T].double() - xd @ wd.t().contiguous()).abs() <= bound).all()
        check_gate(lo[:T], gate, None, idx[:T], w[:T])


def test_route_gate_is_deterministic_and_rows_do_not_mix():
    from split_weight_expert_amd import api
    T, H, E = 500, 1024, 256
    x, wr, _ = route_inputs(T, H, E, "bf16", 9)
    x[7] = float("nan")
    x[8, 3] = float("inf")
    gate = make_gate(8, "sigmoid", 8, 4, 2)
    runs = []
    for _ in range(3):
        idx, w, lo = gate_outputs(T, 8, E)
        api.route_gate(x, wr, gate, lo[:T], idx[:T], w[:T], route_ws(T, H, E, x)[1])
        torch.cuda.synchronize()
        runs.append((idx, w, lo))
    for r in runs[1:]:
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(r, runs[0]))
    idx, w, lo = runs[0]
    assert (idx[7] == -1).all() and (w[7] == 0).all() and lo[7].isnan().all()
    clean = [t for t in range(T) if t not in (7, 8)]
    assert torch.equal(lo[clean].cpu().double(), x[clean].double().cpu() @ wr.double().cpu().t())


# ------------------------------------------------------------------------------------------------ norms

def norm_case(T, H, dt, seed, wdt=None):
    g = gen(seed)
    channel = torch.where(torch.rand(H, generator=g, device=DEV) < 0.05, 12.0, 1.0)
    x = (torch.randn(T, H, generator=g, device=DEV) * 0.5).to(DT[dt])
    r = (torch.randn(T, H, generator=g, device=DEV) * channel).to(DT[dt])
    w = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(DT[wdt or dt])
    return x, r, w


def guarded(T, H, dtype):
    return torch.full((T + 2, H), 77, dtype=dtype, device=DEV)


def check_norm(z, z_err, w, eps, dt, sum_out=None, y=None, q=None, q_scale=None):
    """z: fp64 sums with the absolute error z_err the kernel's fp32 sum may have.

    mean(z^2): each square 1 u, the sum over a row of H at most H/64 + 16 additions deep per element (a thread's
    own elements, then trees) and all terms positive, the division, the addition of eps and 1/sqrt a few u more:
    relative error (H/64 + 24) u of the mean square, half of it on the factor; z's own error enters the mean
    relative to the row's size.  Then two products and the output's rounding."""
    T, H = z.shape
    u = UB16 if dt == "bf16" else U32
    rms = np.sqrt((z * z).mean(1, keepdims=True) + eps)
    n = z / rms * w
    fac = (H / 128 + 24) * U32 + (z_err / np.maximum(rms, 1e-300)).max(1, keepdims=True)
    n_err = np.abs(n) * fac + z_err / rms * np.abs(w) * (1 + 1e-3)
    if sum_out is not None:
        got = sum_out.double().cpu().numpy()
        assert (np.abs(got - z) <= z_err + u * (np.abs(z) + z_err) + 1e-45).all()
    if y is not None:
        got = y.double().cpu().numpy()
        assert (np.abs(got - n) <= n_err + u * (np.abs(n) + n_err) + 1e-40).all()
    if q is not None:
        s = q_scale.double().cpu().numpy()
        c = codecs.e4m3_decode(q.cpu().numpy())
        amax = np.abs(n).reshape(T, H // 128, 128).max(2)
        want = np.where(amax == 0, 1.0, amax / 448)
        e = n_err.reshape(T, H // 128, 128).max(2)
        assert (np.abs(s - want) <= (e + 2 * U32 * amax) / 448 * (1 + 1e-6) + 1e-45).all()
        v = (n.reshape(T, -1, 128) / s[:, :, None]).reshape(T, H)
        v_err = (n_err.reshape(T, -1, 128) / s[:, :, None]).reshape(T, H) + 4 * U32 * np.abs(v)
        half = np.maximum(np.abs(v) + v_err, 2.0 ** -6) * 2.0 ** -4       # half an E4M3 step is at most 2^-4 of the value
        assert (np.abs(c - v) <= half + v_err).all()
        # and the code is the nearest: no neighbouring value is closer by more than the value's error
        vals = np.unique(codecs.E4M3_VALUES[np.isfinite(codecs.E4M3_VALUES)])
        j = np.clip(np.searchsorted(vals, v), 1, len(vals) - 1)
        near = np.minimum(np.abs(v - vals[j]), np.abs(v - vals[j - 1]))
        assert (np.abs(c - v) <= near + 2 * v_err).all()


NORM_SHAPES = [(1, 7168), (1, 1), (3, 7), (5, 8), (64, 128), (65, 256), (7, 1001), (300, 512), (33, 1984), (130, 2048),
               (9, 4104), (17, 7168), (2, 8192), (3, 8200), (2, 16384), (3, 20000), (2, 33001), (2, 40960), (1025, 64), (4, 12289)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_add_rmsnorm(T, H, dt):
    from split_weight_expert_amd import api
    x, r, w = norm_case(T, H, dt, T + H)
    for residual in (r, None):
        z = x.double().cpu().numpy() + (0 if residual is None else r.double().cpu().numpy())
        z_err = U32 * np.abs(z)
        for with_sum, with_y, with_q in ((True, True, True), (False, True, False), (True, False, True), (False, False, True)):
            with_q = with_q and dt == "bf16" and H % 128 == 0
            if not (with_y or with_q):
                continue
            so = guarded(T, H, DT[dt]) if with_sum else None
            y = guarded(T, H, DT[dt]) if with_y else None
            q = guarded(T, H, torch.uint8) if with_q else None
            qs = guarded(T, H // 128, torch.float32) if with_q else None
            cut = lambda t: None if t is None else t[:T]  # noqa: E731
            api.add_rmsnorm(x, residual, w, 1e-6, cut(so), cut(y), cut(q), cut(qs))
            torch.cuda.synchronize()
            for t in (so, y, q, qs):
                assert t is None or (t[T:].float() == 77).all(), "rows behind the last were written"
            check_norm(z, z_err, w.double().cpu().numpy(), 1e-6, dt, cut(so), cut(y), cut(q), cut(qs))


@pytest.mark.parametrize("dt,wdt", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("H", [256, 1001, 7168])
def test_norm_weight_of_the_other_type(dt, wdt, H):
    from split_weight_expert_amd import api
    x, r, w = norm_case(20, H, dt, H, wdt)
    y = torch.empty_like(x)
    api.add_rmsnorm(x, r, w, 1e-5, y=y)
    z = x.double().cpu().numpy() + r.double().cpu().numpy()
    check_norm(z, U32 * np.abs(z), w.double().cpu().numpy(), 1e-5, dt, y=y)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 1001, 1024, 7168, 20000, 40960])
def test_norm_in_place_and_unaligned(dt, H):
    from split_weight_expert_amd import api
    T = 12
    x, r, w = norm_case(T, H, dt, H + 1)
    so, y = torch.empty_like(x), torch.empty_like(x)
    api.add_rmsnorm(x, r, w, 1e-6, so, y)
    for sum_in, y_in in (("r", "x"), ("x", "r"), ("r", None), (None, "x"), (None, "r")):
        bufs = {"x": x.clone(), "r": r.clone(), None: torch.empty_like(x)}
        s2 = bufs[sum_in] if sum_in else torch.empty_like(x)
        y2 = bufs[y_in] if y_in else torch.empty_like(x)
        api.add_rmsnorm(bufs["x"], bufs["r"], w, 1e-6, s2, y2)
        assert torch.equal(s2, so) and torch.equal(y2, y), (sum_in, y_in)
    # element-aligned addresses only
    pad = [torch.zeros(T * H + 3, dtype=DT[dt], device=DEV) for _ in range(4)]
    v = [p[i:i + T * H].view(T, H) for p, i in zip(pad, (1, 2, 3, 1))]
    wp = torch.zeros(H + 1, dtype=DT[dt], device=DEV)
    wp[1:] = w
    v[0].copy_(x)
    v[1].copy_(r)
    api.add_rmsnorm(v[0], v[1], wp[1:], 1e-6, v[2], v[3])
    z = x.double().cpu().numpy() + r.double().cpu().numpy()
    check_norm(z, U32 * np.abs(z), w.double().cpu().numpy(), 1e-6, dt, v[2], v[3])


def test_norm_special_rows():
    """Zero rows, non-finite values (the rows beside them stay clean), tiny and huge values."""
    from split_weight_expert_amd import api
    T, H = 12, 512
    x, _, w = norm_case(T, H, "bf16", 5)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 130] = float("inf")
    x[4] *= 1e-20
    x[5] *= 1e15
    x[6, 128:256] = 0                                     # one group of zeros: scale 1, codes 0
    y, q = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device=DEV)
    qs, so = torch.empty(T, H // 128, device=DEV), torch.empty_like(x)
    api.add_rmsnorm(x, None, w, 1e-6, so, y, q, qs)
    assert torch.equal(so.view(torch.int16), x.view(torch.int16))
    assert (y[1] == 0).all() and (q[1] & 0x7F == 0).all() and (qs[1] == 1).all()
    assert y[2].isnan().all() and qs[2].isnan().all() and ((q[2] & 0x7F) == 0x7F).all()
    # a row with an infinity: factor 0, so the infinity becomes NaN and the rest 0
    assert y[3, 130].isnan() and (torch.cat([y[3, :130], y[3, 131:]]) == 0).all()
    assert qs[3, 1].isnan() and (qs[3, [0, 2, 3]] == 1).all()
    assert (qs[6, 1] == 1).all() and (q[6, 128:256] & 0x7F == 0).all()
    rows = [0, 4, 5, 6, 7, 8, 9, 10, 11]
    z = x[rows].double().cpu().numpy()
    check_norm(z, 0 * z, w.double().cpu().numpy(), 1e-6, "bf16", so[rows], y[rows], q[rows], qs[rows])


def test_norm_codes_are_the_token_quantisers_up_to_its_rounding():
    """With weight 1 and rows whose factor is a power of two, the norm's output is exact in bf16, and its codes and
    scales are bit for bit those of dwdp_quantize_tokens_fp8."""
    from split_weight_expert_amd import api
    T, H = 40, 1024
    g = gen(8)
    x = torch.where(torch.rand(T, H, generator=g, device=DEV) < 0.5, -2.0, 2.0)      # mean square 4: factor 1/2
    x = x.to(torch.bfloat16)
    w = (torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    y, q, qs = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device=DEV), torch.empty(T, H // 128, device=DEV)
    api.add_rmsnorm(x, None, w, 0.0, None, y, q, qs)
    q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
    api.quantize_tokens_fp8(y, q2, qs2)
    assert torch.equal(q, q2) and torch.equal(qs, qs2)


# ------------------------------------------------------------------------------------------------ combine

COMBINE_SHAPES = [(1, 7168, 8, 1), (1, 8, 1, 0), (5, 128, 2, 1), (64, 256, 3, 0), (33, 1984, 6, 1), (17, 7168, 8, 1),
                  (3, 8200, 4, 1), (2, 16384, 2, 0), (2, 40960, 3, 1), (300, 512, 64, 1), (7, 2048, 17, 1), (1030, 64, 2, 1)]


def combine_case(T, H, k, shared, dt, seed):
    g = gen(seed)
    rows = T * (k + shared)
    yp = (torch.randn(rows, H, generator=g, device=DEV) * 0.3).to(DT[dt])
    inv = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    inv[torch.rand(T, k, generator=g, device=DEV) < 0.1] = -1
    if T > 2:
        inv[1] = -1                                       # a token whose every slot was dropped
        inv[2, 0] = rows                                  # out of range: contributes nothing
        inv[2, k - 1] = inv[0, 0]                         # the same row twice
    wt = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
    return yp, inv, wt


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,k,shared", COMBINE_SHAPES)
def test_combine_add_rmsnorm(T, H, k, shared, dt):
    from split_weight_expert_amd import api
    yp, inv, wt = combine_case(T, H, k, shared, dt, T + H + k)
    _, r, w = norm_case(T, H, dt, T + H)
    zc, mag = ol.combine(yp.double().cpu().numpy(), inv.cpu().numpy(), wt.cpu().numpy(), shared)
    for residual in (r, None):
        rn = 0 if residual is None else r.double().cpu().numpy()
        z = zc + rn
        # k products (one rounding each, or none when fused) and k + 2 additions of partial sums
        z_err = (2 * k + 3) * U32 * (mag + np.abs(rn))
        for with_sum, with_y, with_q in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
            with_q = with_q and dt == "bf16" and H % 128 == 0
            if not (with_sum or with_y or with_q):
                continue
            so = guarded(T, H, DT[dt]) if with_sum else None
            y = guarded(T, H, DT[dt]) if with_y else None
            q = guarded(T, H, torch.uint8) if with_q else None
            qs = guarded(T, H // 128, torch.float32) if with_q else None
            cut = lambda t: None if t is None else t[:T]  # noqa: E731
            api.combine_add_rmsnorm(yp, inv, wt, shared, residual, w if with_y or with_q else None, 1e-6, cut(so), cut(y),
                                    cut(q), cut(qs))
            torch.cuda.synchronize()
            for t in (so, y, q, qs):
                assert t is None or (t[T:].float() == 77).all(), "rows behind the last were written"
            check_norm(z, z_err, w.double().cpu().numpy(), 1e-6, dt, cut(so), cut(y), cut(q), cut(qs))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [256, 7168, 40960])
def test_combine_without_residual_is_combine_and_in_place_residuals_work(dt, H):
    from split_weight_expert_amd import api
    T, k = 20, 8
    yp, inv, wt = combine_case(T, H, k, 1, dt, H)
    _, r, w = norm_case(T, H, dt, 3)
    a, b = torch.empty_like(r), torch.empty_like(r)
    api.combine(yp, inv, wt, 1, a)
    api.combine_add_rmsnorm(yp, inv, wt, 1, None, None, 0.0, sum_out=b)
    assert torch.equal(a, b)
    so, y = torch.empty_like(r), torch.empty_like(r)
    api.combine_add_rmsnorm(yp, inv, wt, 1, r, w, 1e-6, so, y)
    r1, y1 = r.clone(), torch.empty_like(r)
    api.combine_add_rmsnorm(yp, inv, wt, 1, r1, w, 1e-6, r1, y1)
    assert torch.equal(r1, so) and torch.equal(y1, y)
    r2, s2 = r.clone(), torch.empty_like(r)
    api.combine_add_rmsnorm(yp, inv, wt, 1, r2, w, 1e-6, s2, r2)
    assert torch.equal(s2, so) and torch.equal(r2, y)


def test_refusals_with_gpu_tensors():
    from split_weight_expert_amd import api
    from split_weight_expert_amd._lib import DwdpError
    x = torch.zeros(4, 256, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(256, device=DEV)
    with pytest.raises(ValueError, match="shape"):
        api.add_rmsnorm(x, x[:3], w, 1e-6, y=torch.empty_like(x))
    with pytest.raises(ValueError, match="type"):
        api.add_rmsnorm(x, None, w, 1e-6, y=torch.empty_like(x).float())
    with pytest.raises(ValueError, match="dense"):
        api.add_rmsnorm(torch.zeros(4, 512, device=DEV)[:, ::2], None, w, 1e-6, y=torch.zeros(4, 256, device=DEV))
    with pytest.raises(ValueError, match="is on cpu"):
        api.add_rmsnorm(x, None, w.cpu(), 1e-6, y=torch.empty_like(x))
    with pytest.raises(DwdpError, match="one of y and q"):
        api.add_rmsnorm(x, None, w, 1e-6)
    with pytest.raises(ValueError, match="shape"):
        api.gate_topk(torch.zeros(4, 8, device=DEV), make_gate(2), torch.zeros(4, 3, dtype=torch.int32, device=DEV),
                      torch.zeros(4, 3, device=DEV))


# ------------------------------------------------------------------------------------------------ streams, graphs

def test_side_stream_and_graph_replays():
    """A captured route_gate -> norm -> boundary, replayed with other inputs in the same buffers and the program's own
    eager work between, gives what the same calls give eagerly; so do calls on a side stream."""
    from split_weight_expert_amd import api
    T, H, E, k = 70, 1024, 64, 4
    gate = make_gate(k, "sigmoid", 8, 4, 2, True, 2.5)
    x, wr, _ = route_inputs(T, H, E, "bf16", 1)
    r = norm_case(T, H, "bf16", 2)[1]
    w = norm_case(T, H, "bf16", 2)[2]
    yp, inv, wt = combine_case(T, H, k, 1, "bf16", 3)
    ws = route_ws(T, H, E, x)[1]

    def outputs():
        return dict(lo=torch.empty(T, E, device=DEV), idx=torch.empty(T, k, dtype=torch.int32, device=DEV),
                    tw=torch.empty(T, k, device=DEV), s=torch.empty_like(r), y=torch.empty_like(r),
                    q=torch.empty(T, H, dtype=torch.uint8, device=DEV), qs=torch.empty(T, H // 128, device=DEV),
                    s2=torch.empty_like(r), y2=torch.empty_like(r))

    def calls(o, wsp, stream=None):
        api.route_gate(x, wr, gate, o["lo"], o["idx"], o["tw"], wsp, stream=stream)
        api.add_rmsnorm(x, r, w, 1e-6, o["s"], o["y"], o["q"], o["qs"], stream=stream)
        api.combine_add_rmsnorm(yp, inv, wt, 1, o["s"], w, 1e-6, o["s2"], o["y2"], stream=stream)

    og, oe, os_ = outputs(), outputs(), outputs()
    calls(og, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(og, ws)
    ws2, ws3 = route_ws(T, H, E, x)[1], route_ws(T, H, E, x)[1]
    side = torch.cuda.Stream()
    for i in range(5):
        x.copy_(route_inputs(T, H, E, "bf16", 10 + i)[0])
        yp.copy_(combine_case(T, H, k, 1, "bf16", 20 + i)[0])
        for t in og.values():
            t.fill_(0)
        graph.replay()
        calls(oe, ws2)
        side.wait_stream(torch.cuda.current_stream())
        calls(os_, ws3, side)
        torch.cuda.synchronize()
        for n in og:
            assert torch.equal(og[n].view(torch.uint8), oe[n].view(torch.uint8)), (i, n)
            assert torch.equal(os_[n].view(torch.uint8), oe[n].view(torch.uint8)), (i, n)


# ------------------------------------------------------------------------------------------------ every lane layout

def special_rows(E, g):
    """Rows where the choice can go wrong: equal and nearly equal logits, masked and non-finite ones."""
    inf, nan = float("inf"), float("nan")
    l = torch.randn(64, E, generator=g, device=DEV)
    l[0] = 0.75
    l[1:5] = torch.randint(0, 3, (4, E), generator=g, device=DEV).float() * 0.5
    l[5:13] = 1.0 + torch.randint(0, 3, (8, E), generator=g, device=DEV).float() * 2.0 ** -23
    l[13] = torch.where(torch.rand(E, generator=g, device=DEV) < 0.5, 0.0, -0.0)
    l[14] = -inf
    l[15] = nan
    l[16] = -inf
    l[16, E - 1] = 0.5
    l[17, : E // 2] = nan
    l[18, E // 3] = inf
    l[19, [0, E - 1]] = inf
    l[20] = torch.finfo(torch.float32).min
    l[21, 1:] = torch.finfo(torch.float32).min
    l[22, ::2] = -inf
    l[23:27] = torch.where(torch.rand(4, E, generator=g, device=DEV) < 0.8, -inf, l[23:27])
    l[27] *= 1e30
    l[28] -= 2000.0
    return l


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top,k", [
    (256, 1, 1, 1, 8), (256, 8, 4, 2, 8), (256, 8, 4, 1, 15), (256, 2, 1, 2, 8), (256, 16, 3, 2, 8), (200, 1, 1, 1, 20), (128, 8, 2, 2, 6),
    (120, 8, 3, 2, 6), (64, 4, 2, 1, 4), (60, 12, 5, 2, 6), (30, 2, 1, 2, 5), (7, 1, 1, 1, 3), (254, 2, 1, 1, 9), (512, 8, 4, 2, 8), (300, 5, 2, 2, 7),
    (1024, 16, 4, 2, 8), (1000, 1, 1, 1, 12), (96, 96, 10, 2, 8)])
def test_few_and_many_tokens_choose_alike(E, groups, kept, top, k, score):
    """The same rows alone and among thousands (other lane layouts): the same experts, the fp64 ones."""
    g = gen(E * 100 + groups * 10 + k)
    l = special_rows(E, g)
    many = l.repeat(36, 1)                              # 2304 rows
    biases = [None, torch.randn(E, generator=g, device=DEV) * 0.05, torch.randint(0, 3, (E,), generator=g, device=DEV).float() * 2.0 ** -22]
    biases[1][E // 2] = -float("inf")
    for balance in biases:
        for renorm in (True, False):
            gate = make_gate(k, score, groups, kept, top, renorm, 1.5)
            i1, w1 = run_gate(l, gate, balance)
            check_gate(l, gate, balance, i1, w1)
            i2, w2 = run_gate(many, gate, balance)
            assert torch.equal(i2.view(36, 64, k), i1.expand(36, 64, k))
            assert torch.equal(w2.view(36, 64, k), w2[:64].expand(36, 64, k))
            check_gate(l, gate, balance, i2[:64], w2[:64])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,top,k", [(256, 1, 1, 1, 8), (256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (255, 5, 2, 2, 14), (130, 1, 1, 1, 4),
                                                 (1024, 16, 4, 2, 8), (999, 1, 1, 1, 32)])
def test_special_rows_among_many_thousands(E, groups, kept, top, k, score):
    """The same with as many tokens as make the chip's issue rate the bound: NaN, infinities, ties, few live experts."""
    g = gen(E + k)
    l = special_rows(E, g)
    many = l.repeat(160, 1)                             # 10240 rows
    b = torch.randn(E, generator=g, device=DEV) * 0.05
    b[E // 2] = -float("inf")
    for balance in (None, b):
        gate = make_gate(k, score, groups, kept, top, True, 1.5)
        i1, w1 = run_gate(many, gate, balance)
        check_gate(l, gate, balance, i1[:64], w1[:64])
        assert torch.equal(i1.view(160, 64, k), i1[:64].expand(160, 64, k))
        assert torch.equal(w1.view(160, 64, k), w1[:64].expand(160, 64, k))


def torch_gate(l, gate, balance):
    """The gate's choice in fp64 by torch (finite logits)."""
    x = l.double()
    s = torch.sigmoid(x) if gate.score == "sigmoid" else torch.softmax(x, 1)
    c = s if balance is None else s + balance.double()
    if gate.topk_groups < gate.n_groups:
        by = c.view(len(c), gate.n_groups, -1)
        val = by.topk(min(gate.group_top, by.shape[2]), 2).values.sum(2)
        keep = torch.zeros_like(val, dtype=torch.bool)
        keep.scatter_(1, val.sort(dim=1, descending=True, stable=True).indices[:, :gate.topk_groups], True)
        c = torch.where(keep[:, :, None], by, -float("inf")).view_as(c)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :gate.k]
    w = s.gather(1, idx)
    return idx.to(torch.int32), (w / w.sum(1, keepdim=True) if gate.renormalize else w) * gate.scale


@pytest.mark.parametrize("E,groups,kept,top,k,score,T", [
    (256, 8, 4, 2, 8, "sigmoid", 60000), (256, 8, 4, 1, 8, "sigmoid", 60000), (256, 1, 1, 1, 8, "sigmoid", 60000),
    (256, 1, 1, 1, 8, "softmax", 60000), (256, 8, 3, 2, 6, "softmax", 60000), (160, 8, 3, 2, 6, "sigmoid", 30000),
    (60, 1, 1, 1, 6, "sigmoid", 60000), (256, 8, 4, 2, 8, "sigmoid", 2000), (512, 8, 4, 2, 8, "sigmoid", 20000),
    (1024, 16, 4, 2, 8, "sigmoid", 10000), (1000, 1, 1, 1, 12, "softmax", 10000)])
def test_close_calls_of_many_tokens(E, groups, kept, top, k, score, T):
    """Enough ordinary tokens that some hundreds have choices, or groups, that fp32 cannot tell apart."""
    g = gen(E + T)
    l = torch.randn(T, E, generator=g, device=DEV) * 1.5
    balance = torch.randn(E, generator=g, device=DEV) * 0.05
    for bal in (balance, None):
        gate = make_gate(k, score, groups, kept, top, True, 2.5)
        idx, w = run_gate(l, gate, bal)
        oi, ow = torch_gate(l, gate, bal)
        assert torch.equal(idx, oi), int((idx != oi).any(1).sum())
        np.testing.assert_array_less((w.double() - ow).abs().cpu().numpy(),
                                     weight_tolerance(l.cpu().numpy(), oi.cpu().numpy(), ow.cpu().numpy()) + 1e-38)


# ------------------------------------------------------------------------------------------------ far offsets

def test_gate_of_more_tokens_than_one_launch_takes():
    """17M tokens: more than 2^20 workgroups of 16 tokens."""
    T = 17_000_000
    l = torch.randn(T, 4, generator=gen(1), device=DEV)
    idx, w = run_gate(l, make_gate(1, "sigmoid", renorm=False))
    assert torch.equal(idx[:, 0].long(), l.argmax(1))
    assert (w[:, 0].double() - torch.sigmoid(l.double().amax(1))).abs().max() < 1e-6


def test_elements_past_32_bits():
    """Arrays of more than 2^31 elements: the last rows are right."""
    from split_weight_expert_amd import api
    T, H, n = 310_000, 7168, 40                       # 2.2e9 elements
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    xs, rs, w = norm_case(n, H, "bf16", 3)
    x[-n:] = xs
    y = torch.empty_like(x)
    q = torch.empty(T, H, dtype=torch.uint8, device=DEV)
    qs = torch.empty(T, H // 128, device=DEV)
    api.add_rmsnorm(x, None, w, 1e-6, None, y, q, qs)
    torch.cuda.synchronize()
    z = xs.double().cpu().numpy()
    check_norm(z, 0 * z, w.double().cpu().numpy(), 1e-6, "bf16", None, y[-n:], q[-n:], qs[-n:])
    assert (y[:1000] == 0).all()
    # y as the permuted rows of 34444 tokens of 8 + 1 rows each, the last of which read the last rows
    k, Tc = 8, 34_444
    inv = torch.arange(Tc * k, device=DEV, dtype=torch.int32).view(Tc, k)
    wt = torch.softmax(torch.randn(Tc, k, generator=gen(4), device=DEV), 1)
    yp = y[: Tc * (k + 1)]
    yp[-3:] = xs[:3]
    yp[Tc * k - 3 * k: Tc * k] = xs[: 3 * k]
    out = torch.empty(Tc, H, dtype=torch.bfloat16, device=DEV)
    api.combine_add_rmsnorm(yp, inv, wt, 1, None, None, 0.0, sum_out=out)
    small = torch.cat([xs[: 3 * k], xs[:3]])
    o1 = torch.empty(3, H, dtype=torch.bfloat16, device=DEV)
    api.combine_add_rmsnorm(small, torch.arange(3 * k, device=DEV, dtype=torch.int32).view(3, k), wt[-3:].contiguous(), 1, None,
                            None, 0.0, sum_out=o1)
    assert torch.equal(out[-3:], o1)
    # and as tokens of the router
    xg, wr, _ = route_inputs(n, H, 256, "bf16", 5)
    x[-n:] = xg
    gate = make_gate(8, "sigmoid", 8, 4, 2)
    idx, tw, lo = gate_outputs(T, 8, 256)
    api.route_gate(x, wr, gate, lo[:T], idx[:T], tw[:T], route_ws(T, H, 256, x)[1])
    torch.cuda.synchronize()
    assert torch.equal(lo[T - n:T].cpu().double(), xg.double().cpu() @ wr.double().cpu().t())
    check_gate(lo[T - n:T], gate, None, idx[T - n:T], tw[T - n:T])
    assert (lo[:1000] == 0).all() and (idx[:1000] == torch.arange(8, device=DEV)).all()


def test_a_stream_and_its_tensors():
    from split_weight_expert_amd import api
    x = torch.zeros(4, 256, device=DEV)

    class Other:
        device_index, cuda_stream = 7, 0
    with pytest.raises(ValueError, match="belongs to GPU 7"):
        api.add_rmsnorm(x, None, x[0], 1e-6, y=torch.empty_like(x), stream=Other())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 9), (7, 15), (130, 17), (67, 129), (40, 263), (33, 511), (600, 513), (9, 2055), (514, 4100), (3, 7161), (4, 16383),
                                 (2, 32767)])
def test_add_rmsnorm_of_widths_no_vector_divides(T, H, dt):
    """The last elements of a row are read and written one by one, and the rows start at odd addresses."""
    from split_weight_expert_amd import api
    x, r, w = norm_case(T, H, dt, T * H)
    for residual in (r, None):
        z = x.double().cpu().numpy() + (0 if residual is None else r.double().cpu().numpy())
        so, y = guarded(T, H, DT[dt]), guarded(T, H, DT[dt])
        api.add_rmsnorm(x, residual, w, 1e-6, so[:T], y[:T])
        torch.cuda.synchronize()
        assert (so[T:] == 77).all() and (y[T:] == 77).all(), "rows behind the last were written"
        check_norm(z, U32 * np.abs(z), w.double().cpu().numpy(), 1e-6, dt, so[:T], y[:T])


def test_scales_of_tiny_rows_stay_normal():
    """amax / 448 below the smallest normal number: the scale is that number, and the codes are finite."""
    from split_weight_expert_amd import api
    T, H = 6, 256
    x = torch.ones(T, H, device=DEV, dtype=torch.bfloat16)
    w = torch.full((H,), 2.0 ** -126, device=DEV)
    w[128:] = 2.0 ** -140
    q, qs = torch.empty(T, H, dtype=torch.uint8, device=DEV), torch.empty(T, H // 128, device=DEV)
    api.add_rmsnorm(x, None, w, 0.0, q=q, q_scale=qs)
    assert (qs == 2.0 ** -126).all()
    c = codecs.e4m3_decode(q.cpu().numpy())
    assert (c[:, :128] == 1).all() and (c[:, 128:] == 0).all()
