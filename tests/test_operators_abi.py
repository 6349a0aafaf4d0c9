"""Branch norms, int8 codes, the balance loss and the gate's gradient without a GPU: bad arguments are rejected before
anything is launched, layouts and sizes are right, and the Python binding refuses wrong tensors."""
import ctypes

import pytest
import torch

lib_mod = pytest.importorskip("split_weight_expert_amd._lib")

FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(0x20000)
FAKE3 = ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10004)
ODDB = ctypes.c_void_p(0x10001)
BAD = lib_mod.DWDP_ERR_INVALID_ARG
INT8, FP8 = lib_mod.INT8, lib_mod.FP8_E4M3


@pytest.fixture(scope="module")
def lib():
    return lib_mod.load()


def expect(rc, lib, needle, code=BAD):
    assert rc == code, (rc, lib.dwdp_last_error())
    assert needle in lib.dwdp_last_error().decode(), lib.dwdp_last_error()


def branch(norm=None, gate=None, nd=1, gd=1, eps=1e-6, scale=1.0, rs=1.0):
    return lib_mod.BranchArgs(norm, gate, nd, gd, eps, scale, rs)


BRANCH_ERRORS = [(dict(nd=2), "dtypes"), (dict(gd=3), "dtypes"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
                 (dict(scale=float("inf")), "scales"), (dict(rs=float("nan")), "scales"),
                 (dict(norm=0x10001), "aligned"), (dict(gate=0x10002, gd=0), "aligned")]


def add(lib, x=FAKE, r=None, dt=1, b=None, tg=None, w=FAKE, wd=1, eps=1e-6, T=4, H=256, s=None, y=FAKE2, q=None, qd=INT8,
        qs=None):
    return lib.dwdp_branch_add_rmsnorm(x, r, dt, None if b is None else ctypes.byref(b), tg, w, wd, eps, T, H, s, y, q, qd,
                                       qs, None)


def combine(lib, x=FAKE, ip=FAKE, tw=FAKE, T=4, k=2, sh=1, H=256, dt=1, r=None, b=None, tg=None, w=FAKE, wd=1, eps=1e-6,
            s=None, y=FAKE2, q=None, qd=INT8, qs=None):
    return lib.dwdp_combine_branch_add_rmsnorm(x, ip, tw, T, k, sh, H, dt, r, None if b is None else ctypes.byref(b), tg, w,
                                               wd, eps, s, y, q, qd, qs, None)


@pytest.mark.parametrize("call", [add, combine])
def test_branch_norms_reject_bad_arguments(lib, call):
    assert ctypes.sizeof(lib_mod.BranchArgs) == 40
    for kw, needle in BRANCH_ERRORS:
        expect(call(lib, b=branch(**kw)), lib, needle)
    for kw, needle in ((dict(dt=2), "dtype"), (dict(wd=2), "w_dtype"), (dict(eps=-1e-6), "eps"),
                       (dict(eps=float("inf")), "eps"), (dict(T=-1), "T out"), (dict(T=1 << 31), "T out"),
                       (dict(H=0), "H must"), (dict(q=FAKE3), "together"), (dict(qs=FAKE3), "together"),
                       (dict(q=FAKE3, qs=FAKE, qd=1), "q_dtype"), (dict(q=FAKE3, qs=FAKE, qd=FP8, H=136), "H % 128"),
                       (dict(q=FAKE3, qs=FAKE, qd=FP8, dt=0), "DWDP_BF16"), (dict(tg=ODDB), "aligned"),
                       (dict(x=None), "NULL" if call is add else "null"), (dict(w=None), "need weight"),
                       (dict(s=FAKE2), "same buffer"), (dict(y=None), "one of sum_out"),
                       (dict(q=ODD, qs=FAKE3), "q: 8"), (dict(q=FAKE3, qs=FAKE2, y=None, r=ODD), "16-byte")):
        expect(call(lib, **kw), lib, needle)
    assert call(lib, T=0, x=None, w=None, y=None) == 0


def test_branch_norms_reject_bad_shapes(lib):
    expect(add(lib, q=FAKE3, qs=FAKE, H=257), lib, "H % 8")
    expect(add(lib, q=FAKE3, qs=FAKE2, y=None, b=branch(norm=0x10004)), lib, "16-byte")
    expect(combine(lib, b=branch(gate=0x10004)), lib, "16-byte")
    for kw, needle in ((dict(k=0), "k must"), (dict(k=65), "k must"), (dict(sh=2), "shared"), (dict(H=100), "multiple of 8"),
                       (dict(T=1 << 30), "T out"), (dict(ip=None), "null"), (dict(tw=None), "null"),
                       (dict(y=FAKE), "y_perm is an output")):
        expect(combine(lib, **kw), lib, needle)


@pytest.mark.parametrize("call", [add, combine])
def test_branch_norms_refuse_overlaps(lib, call):
    step = 1 << 24
    x, r, w, n, g, tg, s, y, q, qs, ip, tw = (step * (i + 1) for i in range(12))
    T, H = 64, 1024
    base = dict(x=x, r=r, w=w, s=s, y=y, q=q, qs=qs, tg=tg, T=T, H=H, b=branch(norm=n, gate=g))
    if call is combine:
        base.update(ip=ip, tw=tw)
    row = H * 2
    for kw in (dict(s=r + row), dict(y=n), dict(y=g - 16), dict(q=tg), dict(qs=tg + T * 4 - 4), dict(qs=q + T * H - 4),
               dict(q=r), dict(y=s + row), dict(s=w), dict(tg=s + 16)):
        expect(call(lib, **dict(base, **kw)), lib, "overlaps")
    # a scale per 128 columns ends behind T * 8 values
    expect(call(lib, **dict(base, qs=w - 1024, qd=FP8)), lib, "overlaps")


def test_quantize_int8_rejects_bad_arguments(lib):
    f = lib.dwdp_quantize_int8
    expect(f(FAKE, 2, 4, 64, FAKE2, FAKE3, None), lib, "dtype")
    expect(f(FAKE, 1, -1, 64, FAKE2, FAKE3, None), lib, "rows")
    expect(f(FAKE, 1, 1 << 31, 64, FAKE2, FAKE3, None), lib, "rows")
    expect(f(FAKE, 1, 4, 0, FAKE2, FAKE3, None), lib, "cols")
    expect(f(FAKE, 1, 4, 60, FAKE2, FAKE3, None), lib, "multiple of 8")
    for a in ((None, FAKE2, FAKE3), (FAKE, None, FAKE3), (FAKE, FAKE2, None)):
        expect(f(a[0], 1, 4, 64, a[1], a[2], None), lib, "null")
    expect(f(ODD, 1, 4, 64, FAKE2, FAKE3, None), lib, "aligned")
    expect(f(FAKE, 1, 4, 64, ODD, FAKE3, None), lib, "aligned")
    expect(f(FAKE, 1, 4, 64, FAKE, FAKE3, None), lib, "overlaps")
    expect(f(FAKE, 1, 4, 64, FAKE2, FAKE2, None), lib, "overlaps")
    assert f(None, 1, 0, 64, None, None, None) == 0


def test_int8_experts_record_workspace_and_limits(lib):
    from split_weight_expert_amd import api
    H, I = 1024, 384
    w2, s13, s2 = api.expert_record_offsets(H, I, INT8)
    assert (w2, s13, s2) == (2 * I * H, 3 * I * H, 3 * I * H + 2 * I * 4)
    rec = api.expert_record_bytes(H, I, INT8)
    assert rec == s2 + H * 4 and rec % 256 == 0
    t = api.fill_expert_table([0x100000], [0, 0], [0, 2], H, I, INT8)
    assert t[1].s13 == 0x100000 + 2 * rec + s13 and t[1].s2 == 0x100000 + 2 * rec + s2
    # the codes, their scales and the fp32 values they are made of
    assert api.workspace_bytes(api.OP_GROUPED_FFN, 64, 2, 8, H, I, INT8, 1) >= 192 * (I * 5 + 4)
    f = lib.dwdp_moe_grouped_ffn
    ws = 1 << 62
    expect(f(FAKE, 9, FAKE, FAKE, None, 128, 256, 128, INT8, FAKE, FAKE, ws, None), lib, "activation scales")
    expect(f(FAKE, 9, FAKE, FAKE, ODDB, 128, 256, 128, INT8, FAKE, FAKE, ws, None), lib, "activation scales")
    for h, i in ((128, 128), (256, 64), (65792, 128), (256, 65664)):
        expect(f(FAKE, 9, FAKE, FAKE, FAKE, 128, h, i, INT8, FAKE, FAKE, ws, None), lib, "H")
    expect(f(FAKE, 9, FAKE, FAKE, FAKE, -1, 65536, 65536, INT8, FAKE, FAKE, ws, None), lib, "rows")
    need = api.workspace_bytes(api.OP_GROUPED_FFN, 64, 2, 8, 256, 128, INT8, 1)
    expect(f(FAKE, 9, FAKE, FAKE, FAKE, 192, 256, 128, INT8, FAKE, FAKE, need - 1, None), lib, "workspace",
           lib_mod.DWDP_ERR_WORKSPACE)
    g = lib.dwdp_moe_grouped_ffn_tokens_static
    expect(g(0, FAKE, 9, FAKE, FAKE, FAKE, FAKE, 64, 1 << 20, 256, 128, INT8, FAKE, None), lib, "static scratch",
           lib_mod.DWDP_ERR_WORKSPACE)
    p = lib.dwdp_pack_weights
    expect(p(FAKE, 32, 64, INT8, FAKE2, None), lib, "int8")
    expect(p(FAKE, 32, 128, 4, FAKE2, None), lib, "DWDP_INT8")
    expect(lib.dwdp_permute(FAKE, 4, 2, 8, 0, FAKE, 1, INT8, 256, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, None), lib,
           "act_dtype")


def balance(lib, l=FAKE, i=FAKE2, T=4, E=8, k=2, score=0, off=None, S=1, c=None, p=None, b=None, z=None, ws=None, n=1 << 40):
    at = [ctypes.c_void_p((a + 8) << 24) for a in range(5)]
    c, p, b, ws = (d if v is None else v for v, d in zip((c, p, b, ws), (at[0], at[1], at[2], at[4])))
    return lib.dwdp_balance_loss(l, i, T, E, k, score, off, S, c, p, b, z, ws, n, None)


def test_balance_loss_rejects_bad_arguments(lib):
    null = ctypes.c_void_p(0)
    for kw, needle in ((dict(score=2), "score"), (dict(k=0), "k must"), (dict(k=33, E=64), "k must"), (dict(k=9), "k must"),
                       (dict(E=0), "E must"), (dict(E=1025), "E must"), (dict(T=-1), "T out"), (dict(T=1 << 30), "T out"),
                       (dict(S=0), "S must"), (dict(S=(1 << 20) + 1, off=FAKE3), "S must"), (dict(S=2), "seq_offsets"),
                       (dict(l=None), "null"), (dict(i=None), "null"), (dict(c=null), "null"), (dict(p=null), "null"),
                       (dict(b=null), "null"), (dict(l=ODDB), "aligned"), (dict(z=ODDB), "aligned"), (dict(off=ODDB), "aligned"),
                       (dict(ws=null), "ws is NULL"), (dict(ws=ODD), "ws is NULL or not"), (dict(c=FAKE), "overlaps"),
                       (dict(p=FAKE2), "overlaps"), (dict(z=FAKE), "overlaps"), (dict(ws=FAKE), "overlaps"),
                       (dict(off=FAKE3, z=FAKE3), "overlaps"), (dict(c=FAKE3, p=FAKE3), "overlaps")):
        expect(balance(lib, **kw), lib, needle)
    need = lib.dwdp_balance_loss_workspace_bytes(4, 8, 1)
    expect(balance(lib, n=need - 1), lib, "workspace", lib_mod.DWDP_ERR_WORKSPACE)
    for bad in ((-1, 8, 1), (1 << 31, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (4, 8, (1 << 20) + 1)):
        assert lib.dwdp_balance_loss_workspace_bytes(*bad) == 0


def test_balance_loss_workspace_grows(lib):
    f = lib.dwdp_balance_loss_workspace_bytes
    ts = sorted({max(0, (1 << p) + d) for p in range(31) for d in (-1, 0, 1, 255)})
    for E, S in ((1, 1), (60, 33), (1024, 1000)):
        sizes = [f(t, E, S) for t in ts]
        assert sizes == sorted(sizes) and f(ts[-1], E, S + 1) >= sizes[-1]
        # chunks of 8 .. 4096 tokens, one more for every sequence: 8 bytes an expert
        assert all(n >= (t // min(max(8, -(-t // 128)), 4096) + S) * E * 8 for t, n in zip(ts, sizes))


def backward(lib, l=FAKE, i=FAKE2, T=4, E=8, g=None, dw=FAKE3, off=None, S=1, c=None, db=None, dz=None,
             d=ctypes.c_void_p(1 << 24)):
    g = lib_mod.GateArgs(0, 2, 1, 1, 1, 1, 1.0) if g is None else g
    return lib.dwdp_gate_backward(l, i, T, E, ctypes.byref(g) if g else None, dw, off, S, c, db, dz, d, None)


def test_gate_backward_rejects_bad_arguments(lib):
    for kw, needle in ((dict(g=False), "gate is NULL"), (dict(g=lib_mod.GateArgs(3, 2, 1, 1, 1, 1, 1.0)), "score"),
                       (dict(g=lib_mod.GateArgs(0, 9, 1, 1, 1, 1, 1.0)), "k must"), (dict(E=0), "E must"),
                       (dict(g=lib_mod.GateArgs(0, 2, 1, 1, 1, 1, float("nan"))), "scale"),
                       (dict(T=-1), "T out"), (dict(T=1 << 30), "T out"), (dict(S=0), "S must"), (dict(S=2), "seq_offsets"),
                       (dict(dw=None), "one of d_w"), (dict(db=FAKE3), "needs counts"), (dict(l=None), "null"),
                       (dict(i=None), "null"), (dict(d=None), "null"), (dict(dw=ODDB), "aligned"), (dict(d=FAKE), "overlaps"),
                       (dict(d=FAKE3), "overlaps"), (dict(c=ctypes.c_void_p(1 << 24)), "overlaps"),
                       (dict(dz=ctypes.c_void_p(1 << 24)), "overlaps")):
        expect(backward(lib, **kw), lib, needle)
    assert backward(lib, T=0, l=None, i=None, d=None) == 0


def test_binding_refuses_wrong_tensors():
    from split_weight_expert_amd import ExpertStore, LayerWeights, MoEBlock, api
    g = api.Gate(k=2)
    x, i, tw = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    b = api.Branch()
    for call in (lambda: api.branch_add_rmsnorm(x, None, b, x[0], 1e-6, y=x),
                 lambda: api.combine_branch_add_rmsnorm(x, torch.zeros(2, 2, dtype=torch.int32), tw, 0, None, b, None, 1e-6),
                 lambda: api.quantize_tokens_int8(x, x.to(torch.int8), x[:, 0]),
                 lambda: api.quantize_weight_int8(x, x.to(torch.int8), x[:, 0]),
                 lambda: api.balance_loss(x, i, g, i, x, x, ws=x), lambda: api.gate_backward(x, i, g, x, tw)):
        with pytest.raises(ValueError, match="current GPU"):
            call()
    with pytest.raises(ValueError, match="gather"):
        MoEBlock(256, 128, 8, 2, 0, "int8", "cpu", gather=True)
    st = ExpertStore(256, 128, INT8, [1], device="cpu")
    w13, w2, s13, s2 = st.views(0, 0)
    assert s13.shape == (256,) and s2.shape == (256,) and w13.numel() == 256 * 256 and w2.numel() == 256 * 128
    good = [torch.zeros(256, 256, dtype=torch.int8), torch.zeros(256), torch.zeros(256, 128, dtype=torch.int8),
            torch.zeros(256)]
    for n, bad in ((0, good[0].float()), (1, torch.zeros(128)), (2, good[2].t()), (3, torch.zeros(256, 1))):
        with pytest.raises(ValueError, match=("w13", "s13", "w2", "s2")[n]):
            st.load_int8(0, 0, *(good[:n] + [bad] + good[n + 1:]))
    with pytest.raises(ValueError, match="not int8"):
        ExpertStore(256, 128, lib_mod.BF16, [1], device="cpu").load_int8(0, 0, *good)
    assert LayerWeights(None, None, None, []).branch is None


def test_pipeline_refuses_a_branch_without_a_norm():
    import unittest.mock as mock
    from types import SimpleNamespace

    from split_weight_expert_amd import DWDPPipeline, LayerWeights, api
    p = object.__new__(DWDPPipeline)           # forward checks its layers before it touches the device
    p.device, p.n_pre, p.rec = torch.device("cpu"), 0, 1
    with mock.patch.object(torch.cuda, "current_stream", return_value=SimpleNamespace()):
        with pytest.raises(ValueError, match="branch needs"):
            p.forward(torch.zeros(2, 4), [LayerWeights(None, None, None, [], branch=api.Branch())])
