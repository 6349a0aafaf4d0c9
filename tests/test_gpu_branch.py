"""Branch norms on the GPU against the fp64 oracle: z = residual_scale residual + scale token_gate gate norm(u), its sum,
its norm, and the norm's E4M3 and int8 codes.

Tolerances.  u is a sum of n = k + shared products in fp32: its error is at most n 2^-23 times the sum of their
magnitudes.  Every element of z takes at most eight more roundings (2^-24 each), and the two factors 1 / sqrt(mean + eps)
a relative error of `steps` roundings, steps = 64 for the sum of squares (at most 32 in a row in a lane, then a tree and
the waves; its terms are positive, so its relative error is theirs, halved by the root), the division and the root.  With M the sum
of magnitudes of z's terms: |dz| <= (n 2^-23 + (8 + steps) 2^-24) M, plus what u's error does to the branch norm's
factor, |n| |du| / |u| (2-norms).  A norm's output adds |y| (|dz| / |z| in 2-norms + steps 2^-24), and a rounding of the
output half a step, eps / 2."""
import numpy as np
import pytest
import torch

from oracle import codecs
from oracle import int8 as o8
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEPS = 64
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_weight_expert_amd import api
    return api


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def norm2(a):
    return np.sqrt((a * a).sum(1, keepdims=True)) + 1e-300


def make(T, H, dtype, seed, norm=True, gate=True, token_gate=True, residual=True, wd=None):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g)
    wd = dtype if wd is None else wd
    return dict(residual=(r(T, H) * 2).to(dtype).to(DEV) if residual else None, weight=(1 + 0.2 * r(H)).to(wd).to(DEV),
                norm=(1 + 0.2 * r(H)).to(wd).to(DEV) if norm else None, gate=(0.5 * r(H)).to(wd).to(DEV) if gate else None,
                token_gate=torch.sigmoid(r(T)).to(DEV) if token_gate else None)


def check(out, u, mag_u, n, c, scale, rs, eps_b, eps, dtype):
    """out: sum / y / q / q_scale as numpy fp64 (or missing); u, mag_u: the exact block output and its terms' magnitudes."""
    norm, gate, tg, res = (f64(c[k]) for k in ("norm", "gate", "token_gate", "residual"))
    z = ol.branch(u, res, norm, eps_b, gate, tg, scale, rs)
    b = ol.branch(u, None, norm, eps_b, gate, tg, scale, rs)
    # the branch's terms' magnitudes: |b| where u's terms do not cancel
    with np.errstate(invalid="ignore", divide="ignore"):
        lift = np.where(u == 0, 0.0, np.abs(b / u))
    mag_b = lift * mag_u
    mag = mag_b + (0 if res is None else np.abs(rs * res))
    du = n * 2 * U * mag_u
    dz = (n * 2 + 8 + STEPS) * U * mag + (np.abs(b) * norm2(du) / norm2(u) if norm is not None else 0)
    half = torch.finfo(dtype).eps / 2
    if "sum" in out:
        assert (np.abs(out["sum"] - z) <= dz + half * np.abs(z) + 1e-38).all()
    w = f64(c["weight"])
    y = ol_norm(z, w, eps)
    dy = np.abs(w) * dz / np.sqrt((z * z).mean(1, keepdims=True) + eps) + np.abs(y) * (norm2(dz) / norm2(z) + STEPS * U)
    if "y" in out:
        assert (np.abs(out["y"] - y) <= dy + half * np.abs(y) + 1e-38).all()
    if "q8" in out:
        s = out["s8"].repeat(128, 1)
        amax = np.abs(y).reshape(len(y), -1, 128).max(2)
        dmax = dy.reshape(len(y), -1, 128).max(2)
        assert (np.abs(out["s8"] - amax / 448) <= dmax / 448 + 4 * U * amax / 448).all()
        # E4M3: half a step is 2^-4 of the value, or 2^-10 scales below the normal range
        assert (np.abs(out["q8"] * s - y) <= dy + np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) * (1 + 8 * U) + dy).all()
    if "qi" in out:
        s = out["si"][:, None]
        amax, dmax = np.abs(y).max(1, keepdims=True), dy.max(1, keepdims=True)
        assert (np.abs(s - amax / 127) <= dmax / 127 + 4 * U * amax / 127).all()
        assert (np.abs(out["qi"] * s - y) <= 0.5 * s * (1 + 256 * 2 * U) + dy).all()
        assert np.abs(out["qi"]).max(1).min() == 127


def ol_norm(z, w, eps):
    return z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * w


def outputs(T, H, dtype, kinds):
    """Buffers with a row of sentinels behind each."""
    o = {}
    if "sum" in kinds:
        o["sum_out"] = torch.full((T + 1, H), 7.0, dtype=dtype, device=DEV)
    if "y" in kinds:
        o["y"] = torch.full((T + 1, H), 7.0, dtype=dtype, device=DEV)
    if "fp8" in kinds:
        o["q"] = torch.full((T + 1, H), 99, dtype=torch.uint8, device=DEV)
        o["q_scale"] = torch.full((T + 1, H // 128), 7.0, device=DEV)
    if "int8" in kinds:
        o["q"] = torch.full((T + 1, H), 99, dtype=torch.int8, device=DEV)
        o["q_scale"] = torch.full((T + 1,), 7.0, device=DEV)
    return o


def results(o, T, kinds):
    for t in o.values():
        assert (t[T:].double() == (99 if t.dtype in (torch.uint8, torch.int8) else 7)).all(), "written behind the last row"
    r = {}
    if "sum" in kinds:
        r["sum"] = f64(o["sum_out"][:T])
    if "y" in kinds:
        r["y"] = f64(o["y"][:T])
    if "fp8" in kinds:
        r["q8"], r["s8"] = codecs.e4m3_decode(o["q"][:T].cpu().numpy()), f64(o["q_scale"][:T])
    if "int8" in kinds:
        r["qi"], r["si"] = f64(o["q"][:T]), f64(o["q_scale"][:T])
    return r


ADD = [(1, 8, "f32", "sum y int8"), (3, 1, "f32", "sum y"), (5, 7, "bf16", "sum y"), (70, 100, "bf16", "sum y"),
       (9, 128, "bf16", "sum y fp8"), (9, 248, "bf16", "int8"), (300, 256, "bf16", "y fp8"), (2, 512, "bf16", "sum y int8"),
       (33, 1001, "f32", "sum y"), (17, 2048, "bf16", "sum int8"), (5, 7168, "bf16", "sum y fp8"), (1, 7168, "bf16", "sum y int8"),
       (2049, 2056, "bf16", "sum y int8"), (7, 8200, "f32", "sum y int8"), (3, 16384, "bf16", "sum y fp8"),
       (3, 20000, "bf16", "sum y int8"), (2, 32768, "bf16", "int8"), (2, 33001, "f32", "sum y"), (3, 40960, "bf16", "sum y int8"),
       (2, 40960, "bf16", "sum y fp8")]


@pytest.mark.parametrize("T,H,dt,kinds", ADD)
def test_branch_add(api, T, H, dt, kinds):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    kinds = kinds.split()
    c = make(T, H, dtype, T * 7 + H)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).to(dtype).to(DEV)
    b = api.Branch(norm=c["norm"], eps=1e-5, gate=c["gate"], scale=0.4, residual_scale=1.3)
    o = outputs(T, H, dtype, kinds)
    api.branch_add_rmsnorm(x, c["residual"], b, c["weight"], 1e-6, token_gate=c["token_gate"], **{k: t[:T] for k, t in o.items()})
    u = f64(x)
    check(results(o, T, kinds), u, np.abs(u), 0, c, 0.4, 1.3, 1e-5, 1e-6, dtype)


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("gate,token_gate,residual", [(0, 0, 0), (1, 0, 1), (0, 1, 1), (1, 1, 0)])
def test_every_part_may_be_missing(api, norm, gate, token_gate, residual):
    T, H = 6, 640
    c = make(T, H, torch.bfloat16, 5, norm, gate, token_gate, residual, wd=torch.float32)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    b = api.Branch(norm=c["norm"], gate=c["gate"], scale=-2.0, residual_scale=0.0 if token_gate else -1.0)
    o = outputs(T, H, torch.bfloat16, ["sum", "y", "int8"])
    api.branch_add_rmsnorm(x, c["residual"], b, c["weight"], 1e-6, token_gate=c["token_gate"], **{k: t[:T] for k, t in o.items()})
    check(results(o, T, ["sum", "y", "int8"]), f64(x), np.abs(f64(x)), 0, c, -2.0, b.residual_scale, 1e-6, 1e-6, torch.bfloat16)


COMBINE = [(1, 8, 1, 0, "f32", "sum y"), (4, 136, 3, 1, "bf16", "sum y int8"), (65, 256, 6, 1, "bf16", "sum y fp8"),
           (3, 1024, 64, 0, "bf16", "sum y int8"), (2, 7168, 8, 1, "bf16", "sum y fp8"), (300, 7168, 8, 1, "bf16", "y int8"),
           (5, 4096, 11, 1, "f32", "sum y int8"), (2, 16384, 2, 1, "bf16", "sum y fp8"), (2, 17408, 2, 1, "bf16", "sum y int8"),
           (3, 17408, 3, 0, "f32", "sum y")]


@pytest.mark.parametrize("T,H,k,shared,dt,kinds", COMBINE)
def test_combine_branch(api, T, H, k, shared, dt, kinds):
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    kinds = kinds.split()
    g = torch.Generator().manual_seed(T + H)
    c = make(T, H, dtype, T + H + 1)
    yp = torch.randn(T * (k + shared), H, generator=g).to(dtype)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    if T > 2:
        inv[1, 0] = -1
        inv[2] = -1                          # a token whose slots are all dropped
        inv[0, 0] = T * (k + shared)         # out of range
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    u, mag = np.zeros((T, H)), np.zeros((T, H))
    y64 = yp.double().numpy()
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < T * (k + shared):
                u[t] += float(w[t, j]) * y64[inv[t, j]]
                mag[t] += np.abs(float(w[t, j]) * y64[inv[t, j]])
        if shared:
            u[t] += y64[T * k + t]
            mag[t] += np.abs(y64[T * k + t])
    b = api.Branch(norm=c["norm"], eps=1e-5, gate=c["gate"], scale=0.7, residual_scale=1.1)
    o = outputs(T, H, dtype, kinds)
    api.combine_branch_add_rmsnorm(yp.to(DEV), inv.to(DEV), w.to(DEV), shared, c["residual"], b, c["weight"], 1e-6,
                                   token_gate=c["token_gate"], **{n: t[:T] for n, t in o.items()})
    check(results(o, T, kinds), u, mag, k + shared, c, 0.7, 1.1, 1e-5, 1e-6, dtype)


def test_a_plain_branch_is_the_norm_without_one(api):
    """Without norm and gates and with scales of 1 the results are those of the calls without a branch, bit for bit."""
    g = torch.Generator().manual_seed(2)
    for T, H, dtype in ((3, 7168, torch.bfloat16), (50, 1001, torch.float32), (2, 40000, torch.bfloat16)):
        x, r = (torch.randn(T, H, generator=g).to(dtype).to(DEV) for _ in range(2))
        w = torch.randn(H, generator=g).to(DEV)
        a, b = ([torch.empty_like(x) for _ in range(2)] for _ in range(2))
        api.add_rmsnorm(x, r, w, 1e-6, sum_out=a[0], y=a[1])
        api.branch_add_rmsnorm(x, r, None, w, 1e-6, sum_out=b[0], y=b[1])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        k = 3
        yp = torch.randn(T * (k + 1), 1024, generator=g).to(dtype).to(DEV)
        inv = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k).to(DEV)
        tw, w = torch.rand(T, k, generator=g).to(DEV), w[:1024].contiguous() if H >= 1024 else torch.ones(1024, device=DEV)
        r = torch.randn(T, 1024, generator=g).to(dtype).to(DEV)
        a, b = ([torch.empty_like(r) for _ in range(2)] for _ in range(2))
        api.combine_add_rmsnorm(yp, inv, tw, 1, r, w, 1e-6, sum_out=a[0], y=a[1])
        api.combine_branch_add_rmsnorm(yp, inv, tw, 1, r, api.Branch(), w, 1e-6, sum_out=b[0], y=b[1])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H", [256, 7168, 40960])
def test_in_place_and_repeated(api, H):
    T = 5
    c = make(T, H, torch.bfloat16, 3)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).bfloat16().to(DEV)
    b = api.Branch(norm=c["norm"], gate=c["gate"], scale=0.3)

    def run(x, r, **kw):
        q, qs = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        api.branch_add_rmsnorm(x, r, b, c["weight"], 1e-6, q=q, q_scale=qs, token_gate=c["token_gate"], **kw)
        return q, qs
    s, y = torch.empty_like(x), torch.empty_like(x)
    want = (*run(x, c["residual"], sum_out=s, y=y), s, y)
    for _ in range(3):
        xi, ri = x.clone(), c["residual"].clone()
        q, qs = run(xi, ri, sum_out=ri, y=xi)
        assert all(torch.equal(a, w) for a, w in zip((q, qs, ri, xi), want))


def test_zero_and_nonfinite_rows(api):
    """A zero branch output keeps the residual; a NaN or an infinity stays in its row, whose int8 scale is NaN."""
    T, H = 6, 512
    c = make(T, H, torch.float32, 9, token_gate=False)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(DEV)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    r = c["residual"]
    r[4], x[4] = 0, 0
    o = outputs(T, H, torch.float32, ["sum", "y", "int8"])
    api.branch_add_rmsnorm(x, r, api.Branch(norm=c["norm"], gate=c["gate"]), c["weight"], 1e-6, **{k: t[:T] for k, t in o.items()})
    s, y, q, qs = (o[k][:T] for k in ("sum_out", "y", "q", "q_scale"))
    assert torch.equal(s[1], r[1]) and torch.isnan(s[2]).all() and not torch.isfinite(s[3, 7])
    assert torch.isnan(qs[2]) and torch.isnan(qs[3]) and (q[2] == 0).all() and (q[3] == 0).all()
    assert (s[4] == 0).all() and (y[4] == 0).all() and (q[4] == 0).all() and qs[4] == 1
    keep = torch.tensor([0, 1, 5], device=DEV)
    assert torch.isfinite(y[keep]).all() and (q[keep].abs().amax(1) == 127).all()


def test_int8_codes_are_those_of_the_quantiser(api):
    """int8 codes come from the unrounded norm: for fp32 outputs they are the quantiser's of y."""
    T, H = 40, 2048
    c = make(T, H, torch.float32, 11)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = torch.empty_like(x)
    q, q2 = (torch.empty(T, H, dtype=torch.int8, device=DEV) for _ in range(2))
    s, s2 = (torch.empty(T, device=DEV) for _ in range(2))
    api.branch_add_rmsnorm(x, c["residual"], api.Branch(norm=c["norm"]), c["weight"], 1e-6, y=y, q=q, q_scale=s)
    api.quantize_tokens_int8(y, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    want, ws = o8.rows(y.cpu().numpy())
    assert np.array_equal(want, q.cpu().numpy()) and np.array_equal(ws, s.cpu().numpy())


def test_binding_refuses_wrong_tensors_on_the_gpu(api):
    T, H = 4, 256
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, device=DEV)
    y = torch.empty_like(x)
    cases = [(dict(branch=api.Branch(norm=w[:128])), "branch.norm"), (dict(branch=api.Branch(gate=w.half())), "branch.gate"),
             (dict(branch=api.Branch(gate=w.cpu())), "branch.gate"), (dict(token_gate=torch.ones(T + 1, device=DEV)), "token_gate"),
             (dict(token_gate=torch.ones(T, 1, device=DEV)), "token_gate"), (dict(residual=x.float()), "residual"),
             (dict(q=torch.empty(T, H, dtype=torch.int16, device=DEV)), "q must"),
             (dict(q=torch.empty(T, H, dtype=torch.int8, device=DEV), q_scale=torch.empty(T, 2, device=DEV)), "q_scale"),
             (dict(q=torch.empty(T, H, dtype=torch.uint8, device=DEV), q_scale=torch.empty(T, device=DEV)), "q_scale")]
    for kw, needle in cases:
        a = dict(dict(residual=None, branch=None, weight=w, eps=1e-6, y=y), **kw)
        with pytest.raises(ValueError, match=needle):
            api.branch_add_rmsnorm(x, **a)
        with pytest.raises(ValueError, match=needle):
            api.combine_branch_add_rmsnorm(torch.zeros(2 * T, H, dtype=torch.bfloat16, device=DEV),
                                           torch.zeros(T, 2, dtype=torch.int32, device=DEV), torch.zeros(T, 2, device=DEV), 0, **a)
    api.branch_add_rmsnorm(x[:0], None, None, w, 1e-6, y=y[:0])
