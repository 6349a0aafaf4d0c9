"""include/dwdp_layer.h without a GPU: every declared symbol is exported and bound, bad arguments are rejected
before anything is launched, and the Python binding refuses wrong tensors."""
import copy
import ctypes
import os
import pickle
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dwdp_layer.h")

lib_mod = pytest.importorskip("split_weight_expert_amd._lib")

FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced: validation fails first
FAKE2 = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)
ODDB = ctypes.c_void_p(0x10001)
BAD = lib_mod.DWDP_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return lib_mod.load()


def expect(rc, lib, needle, code=BAD):
    assert rc == code, (rc, lib.dwdp_last_error())
    assert needle in lib.dwdp_last_error().decode(), lib.dwdp_last_error()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(dwdp_[a-z0-9_]+)\s*\(", text))
    assert names == set(lib_mod.LAYER_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n
    assert ctypes.sizeof(lib_mod.GateArgs) == 28


def gate(**kw):
    a = dict(score=1, k=8, n_groups=8, topk_groups=4, group_top=2, renormalize=1, scale=1.0)
    a.update(kw)
    return lib_mod.GateArgs(**a)


GATE_ERRORS = [
    (dict(score=2), 256, "score"), (dict(k=0), 256, "k must"), (dict(k=33), 256, "k must"), (dict(k=9), 8, "k must"),
    (dict(n_groups=0), 256, "n_groups"), (dict(n_groups=7), 256, "n_groups"), (dict(n_groups=512), 256, "n_groups"),
    (dict(topk_groups=0), 256, "topk_groups"), (dict(topk_groups=9), 256, "topk_groups"),
    (dict(n_groups=64, topk_groups=1), 256, "experts of topk_groups"), (dict(group_top=0), 256, "group_top"),
    (dict(group_top=3), 256, "group_top"), (dict(renormalize=2), 256, "renormalize"),
    (dict(scale=float("inf")), 256, "scale"), (dict(scale=float("nan")), 256, "scale"), (dict(), 0, "E must"),
    (dict(), 1032, "E must"),
]


@pytest.mark.parametrize("kw,E,needle", GATE_ERRORS)
def test_bad_gates_are_rejected(lib, kw, E, needle):
    g = ctypes.byref(gate(**kw))
    expect(lib.dwdp_gate_topk(FAKE, None, 4, E, g, FAKE, FAKE, None), lib, needle)
    expect(lib.dwdp_route_gate(FAKE, FAKE, 1, None, None, 4, 256, E, g, FAKE, FAKE, FAKE, FAKE, 1 << 40, None), lib, needle)


def test_gate_and_route_reject_bad_arguments(lib):
    g = ctypes.byref(gate())
    f = lib.dwdp_gate_topk
    expect(f(FAKE, None, 4, 256, None, FAKE, FAKE, None), lib, "gate is NULL")
    expect(f(None, None, 4, 256, g, FAKE, FAKE, None), lib, "null")
    expect(f(FAKE, None, 4, 256, g, None, FAKE, None), lib, "null")
    expect(f(FAKE, None, 4, 256, g, FAKE, None, None), lib, "null")
    expect(f(FAKE, None, -1, 256, g, FAKE, FAKE, None), lib, "T out of range")
    expect(f(FAKE, None, 1 << 31, 256, g, FAKE, FAKE, None), lib, "T out of range")
    expect(f(ODDB, None, 4, 256, g, FAKE, FAKE, None), lib, "aligned")
    assert f(None, None, 0, 256, g, None, None, None) == 0

    def r(x=FAKE, w=FAKE, dt=1, T=4, H=256, E=256, lo=FAKE, i=FAKE, tw=FAKE, ws=FAKE, n=1 << 40):
        return lib.dwdp_route_gate(x, w, dt, None, None, T, H, E, g, lo, i, tw, ws, n, None)
    expect(r(dt=2), lib, "in_dtype")
    expect(r(H=100), lib, "H % 64")
    expect(r(H=8, dt=0), lib, "H % 16")
    expect(r(H=0), lib, "H must")
    expect(r(x=None), lib, "null")
    expect(r(lo=None), lib, "null")
    expect(r(x=ODD), lib, "aligned")
    expect(r(w=ODD), lib, "aligned")
    expect(r(T=-1), lib, "T out of range")
    assert r(T=0, x=None, w=None, lo=None, i=None, tw=None, ws=None, n=0) == 0
    # 2^30 tokens of 1024 experts: no launch holds the router's tiles
    need = lib.dwdp_route_gate_workspace_bytes(1 << 30, 64, 1024, 1)
    g1 = ctypes.byref(gate(n_groups=1, topk_groups=1))
    expect(lib.dwdp_route_gate(FAKE, FAKE, 1, None, None, 1 << 30, 64, 1024, g1, FAKE, FAKE, FAKE, FAKE, need, None), lib,
           "too large")


def test_route_gate_needs_the_workspace_it_names(lib):
    g = ctypes.byref(gate())
    for T, H, E, dt in ((1, 7168, 256, 1), (64, 7168, 256, 1), (8192, 7168, 256, 1), (300, 512, 256, 0)):
        need = lib.dwdp_route_gate_workspace_bytes(T, H, E, dt)
        if need == 0:
            continue
        a = [FAKE, FAKE, dt, None, None, T, H, E, g, FAKE, FAKE, FAKE]
        expect(lib.dwdp_route_gate(*a, FAKE, need - 1, None), lib, "workspace", lib_mod.DWDP_ERR_WORKSPACE)
        expect(lib.dwdp_route_gate(*a, None, need, None), lib, "ws is NULL")
        expect(lib.dwdp_route_gate(*a, ODD, need, None), lib, "ws is NULL or not")
    for bad in ((-1, 7168, 256, 1), (64, 0, 256, 1), (64, 7168, 0, 1), (64, 7168, 256, 2), (0, 7168, 256, 1)):
        assert lib.dwdp_route_gate_workspace_bytes(*bad) == 0


def test_add_rmsnorm_rejects_bad_arguments(lib):
    def f(x=FAKE, r=None, dt=1, w=FAKE, wd=1, eps=1e-6, T=4, H=256, s=None, y=FAKE2, q=None, qs=None):
        return lib.dwdp_add_rmsnorm(x, r, dt, w, wd, eps, T, H, s, y, q, qs, None)
    expect(f(dt=2), lib, "dtype")
    expect(f(wd=2), lib, "w_dtype")
    expect(f(eps=-1e-6), lib, "eps")
    expect(f(eps=float("nan")), lib, "eps")
    expect(f(T=-1), lib, "T out")
    expect(f(T=1 << 31), lib, "T out")
    expect(f(H=0), lib, "H must")
    expect(f(q=FAKE), lib, "together")
    expect(f(qs=FAKE), lib, "together")
    expect(f(q=FAKE, qs=FAKE, H=200), lib, "H % 128")
    expect(f(q=FAKE, qs=FAKE, dt=0), lib, "DWDP_BF16")
    expect(f(q=ODD, qs=FAKE), lib, "q: 8")
    expect(f(q=FAKE, qs=FAKE, x=ODD), lib, "16-byte")
    expect(f(x=None), lib, "NULL")
    expect(f(w=None), lib, "NULL")
    expect(f(y=None), lib, "one of y and q")
    expect(f(s=FAKE2), lib, "same buffer")
    expect(f(x=ODDB), lib, "aligned")
    expect(f(w=ctypes.c_void_p(0x10002), wd=0), lib, "aligned")
    assert f(T=0, x=None, w=None, y=None) == 0


def test_combine_add_rmsnorm_rejects_bad_arguments(lib):
    def f(yp=FAKE, ip=FAKE, tw=FAKE, T=4, k=2, sh=1, H=256, dt=1, r=FAKE, w=FAKE, wd=1, eps=1e-6, s=FAKE2, y=None,
          q=None, qs=None):
        return lib.dwdp_combine_add_rmsnorm(yp, ip, tw, T, k, sh, H, dt, r, w, wd, eps, s, y, q, qs, None)
    expect(f(dt=2), lib, "dtype")
    expect(f(wd=3), lib, "w_dtype")
    expect(f(eps=float("inf")), lib, "eps")
    expect(f(k=0), lib, "k must")
    expect(f(k=65), lib, "k must")
    expect(f(sh=2), lib, "shared")
    expect(f(T=-1), lib, "T out")
    expect(f(T=1 << 30, k=2), lib, "T out")
    expect(f(H=100), lib, "multiple of 8")
    expect(f(q=FAKE2, qs=FAKE, H=200), lib, "H % 128")
    expect(f(q=FAKE2), lib, "together")
    expect(f(q=FAKE2, qs=FAKE, dt=0), lib, "DWDP_BF16")
    expect(f(yp=None), lib, "null")
    expect(f(ip=None), lib, "null")
    expect(f(tw=None), lib, "null")
    expect(f(s=None), lib, "one of sum_out")
    expect(f(y=ctypes.c_void_p(0x30000), w=None), lib, "need weight")
    expect(f(y=FAKE2), lib, "same buffer")
    expect(f(s=FAKE), lib, "y_perm is an output")
    expect(f(r=ODD), lib, "aligned")
    assert f(T=0, yp=None, ip=None, tw=None, s=None) == 0


def _at(base, step=1 << 24):
    """Distinct made-up addresses, far enough apart for the sizes below."""
    return ctypes.c_void_p(base * step)


def test_overlapping_buffers_are_refused(lib):
    g = ctypes.byref(gate())
    T, H, E = 64, 1024, 256
    x, w, bias, bal, lo, i, tw, ws, r, s, y, q, qs = (_at(n + 1) for n in range(13))

    def inside(p, off):
        return ctypes.c_void_p(p.value + off)
    f = lib.dwdp_gate_topk
    for args in ((lo, bal, lo, tw), (lo, bal, i, inside(lo, T * E * 4 - 4)), (lo, bal, i, i), (lo, bal, bal, tw),
                 (lo, bal, inside(tw, T * 8 * 4 - 4), tw)):
        expect(f(args[0], args[1], T, E, g, args[2], args[3], None), lib, "overlaps")

    need = lib.dwdp_route_gate_workspace_bytes(T, H, E, 1)
    assert need > 0
    base = dict(x=x, w=w, bias=bias, bal=bal, lo=lo, i=i, tw=tw, ws=ws)

    def route(**kw):
        a = dict(base, **kw)
        return lib.dwdp_route_gate(a["x"], a["w"], 1, a["bias"], a["bal"], T, H, E, g, a["lo"], a["i"], a["tw"], a["ws"],
                                   need, None)
    for kw in (dict(lo=x), dict(lo=inside(w, E * H * 2 - 4)), dict(i=lo), dict(tw=i), dict(ws=x), dict(ws=lo), dict(i=ws),
               dict(tw=bal), dict(lo=bias), dict(x=inside(ws, need - 16))):
        expect(route(**kw), lib, "overlaps")

    nbase = dict(x=x, r=r, w=w, s=s, y=y, q=q, qs=qs)

    def norm(**kw):
        a = dict(nbase, **kw)
        return lib.dwdp_add_rmsnorm(a["x"], a["r"], 1, a["w"], 1, 1e-6, T, H, a["s"], a["y"], a["q"], a["qs"], None)

    def combine(**kw):
        a = dict(nbase, ip=i, tw=tw, **kw)
        return lib.dwdp_combine_add_rmsnorm(a["x"], a["ip"], a["tw"], T, 8, 1, H, 1, a["r"], a["w"], 1, 1e-6, a["s"], a["y"],
                                            a["q"], a["qs"], None)
    row = H * 2
    for kw in (dict(s=inside(r, row)), dict(y=inside(r, -row)), dict(q=r), dict(q=x), dict(qs=x), dict(qs=w), dict(y=w),
               dict(q=s), dict(y=inside(s, row)), dict(qs=inside(q, T * H - 4)), dict(w=inside(y, row))):
        expect(norm(**kw), lib, "overlaps")
        expect(combine(**kw), lib, "overlaps" if kw.get("q") is not x else "is an output")
    expect(norm(s=inside(x, row)), lib, "overlaps")
    for kw in (dict(s=inside(x, 9 * T * row - row)), dict(y=i), dict(qs=tw)):
        expect(combine(**kw), lib, "overlaps")


def test_gate_object():
    from split_weight_expert_amd import api
    g = api.Gate(k=8, score="sigmoid", n_groups=8, topk_groups=4, group_top=2, scale=2.5)
    for h in (copy.deepcopy(g), pickle.loads(pickle.dumps(g))):
        assert h == g and bytes(h._c) == bytes(g._c)
    with pytest.raises(ValueError):
        api.Gate(k=8, score="relu")
    with pytest.raises(ValueError, match="32-bit"):
        api.Gate(k=8, n_groups=(1 << 32) + 1)


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    from split_weight_expert_amd import MoEBlock, api
    g = api.Gate(k=2)
    x, w = torch.zeros(4, 64), torch.zeros(8, 64)
    i, tw, lo = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="current GPU"):
        api.route_gate(x, w, g, lo, i, tw)
    with pytest.raises(ValueError, match="current GPU"):
        api.gate_topk(lo, g, i, tw)
    with pytest.raises(ValueError, match="current GPU"):
        api.add_rmsnorm(x, None, x[0], 1e-6, y=x)
    with pytest.raises(ValueError, match="current GPU"):
        api.combine_add_rmsnorm(x, torch.zeros(2, 2, dtype=torch.int32), tw, 0, None, None, 1e-6, sum_out=x)
    with pytest.raises(ValueError, match="2 dimensions"):
        api.gate_topk(lo[0], g, i, tw)
    with pytest.raises(ValueError, match="columns"):       # 2^32 + 8 columns would be 8 to the library
        api.add_rmsnorm(torch.empty(1, (1 << 32) + 8, device="meta"), None, x[0], 1e-6, y=x)
    with pytest.raises(ValueError, match="the block is for"):
        MoEBlock(256, 128, 8, 3, 0, "f32", "cpu", gate=g)


def test_tensor_checks():
    """The check every tensor of these calls goes through (on CPU tensors: it reads no device memory)."""
    from split_weight_expert_amd import api
    cpu = -1                                   # a CPU tensor's device number
    f32 = (torch.float32,)
    t = torch.zeros(4, 8)
    assert api._check("t", None, (4, 8), f32, cpu) is None
    assert api._check("t", t, (4, 8), f32, cpu) == t.data_ptr()
    for bad, match in ((torch.zeros(4, 9), "shape"), (torch.zeros(4, 8, dtype=torch.float64), "type"),
                       (torch.zeros(8, 4).t(), "dense"), (torch.zeros(4, 16)[:, ::2], "dense"),
                       ):
        with pytest.raises(ValueError, match=match):
            api._check("t", bad, (4, 8), f32, cpu)
    with pytest.raises(ValueError, match="is on cpu, not on GPU 0"):
        api._check("t", t, (4, 8), f32, 0)


def test_pipeline_refuses_mixed_norms():
    from types import SimpleNamespace

    from split_weight_expert_amd import DWDPPipeline, LayerWeights
    p = object.__new__(DWDPPipeline)           # forward checks its layers before it touches the device
    p.device, p.n_pre, p.rec = torch.device("cpu"), 0, 1
    lw = [LayerWeights(None, None, None, [], norm=n) for n in (torch.ones(4), None)]
    import unittest.mock as mock
    with mock.patch.object(torch.cuda, "current_stream", return_value=SimpleNamespace()):
        with pytest.raises(ValueError, match="some layers have a norm"):
            p.forward(torch.zeros(2, 4), lw)
        with pytest.raises(ValueError, match="chain"):
            p.forward(torch.zeros(2, 4), lw[:1], chain=False)


def test_one_workspace_serves_every_batch(lib):
    """The size is not monotonic in T, but bounded: a buffer of the bound is taken for every batch."""
    from split_weight_expert_amd import api
    text = open(HEADER).read()
    assert "DWDP_ROUTE_GATE_WORKSPACE_MAX ((size_t)32 << 20)" in text and api.ROUTE_GATE_WORKSPACE_MAX == 32 << 20
    need = [lib.dwdp_route_gate_workspace_bytes(T, 7168, 256, 1) for T in (64, 8192, 10000, 16384, 32768)]
    assert need[1] > need[2] > 0 and need[4] == 0
    ts = sorted({min(max(b + d, 1), 1 << 21) for p in range(22) for b in (1 << p, 5 << p) for d in (-1, 0, 1)})
    for dt, hs in ((1, (64, 1984, 7168, 16384, 1 << 20)), (0, (16, 1040, 7168, 1 << 20))):
        for H in hs:
            for E in (1, 16, 60, 64, 65, 128, 129, 256, 257, 320, 512, 513, 1000, 1024):
                for T in ts:
                    assert lib.dwdp_route_gate_workspace_bytes(T, H, E, dt) <= api.ROUTE_GATE_WORKSPACE_MAX, (T, H, E, dt)
