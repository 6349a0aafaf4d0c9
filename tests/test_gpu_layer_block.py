"""The gate, the norms and the layer boundary inside the block and the pipeline, against the oracle.

MoEBlock(gate=...) with a sigmoid, group-limited gate; and a pipeline of pre-norm residual layers,
h_{l+1} = h_l + block_l(norm_l(h_l)): every layer's normed input, its routing (whole numbers) and its output are
checked against the oracle applied to the GPU's own input of that step.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import layer as ol
from oracle import moe as omoe
from synth.configs import shrink
from tests.gpu_util import HostLayer, assert_close, need_gpu, to_np, upload_layer
from tests.test_gpu_layer import U32, check_norm
from tests.test_gpu_pipeline import SLEEP, build_layers

pytestmark = pytest.mark.gpu

DEV = "cuda"
CASES = {
    "f32": ("tiny_f32", dict(T=96, H=256, I=128, E=8, k=2, shared=1, n_local=3, n_sources=1)),
    "bf16": ("prefill8k_bf16", dict(T=160, H=512, I=256, E=12, k=3, shared=1, n_local=4, n_sources=2)),
    "fp8": ("prefill16k_fp8", dict(T=160, H=512, I=256, E=12, k=3, shared=1, n_local=4, n_sources=2)),
}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def make_gate(cfg):
    from split_weight_expert_amd import api
    return api.Gate(k=cfg.k, score="sigmoid", n_groups=4, topk_groups=2, group_top=2, scale=1.5)


def oracle_gate(gate, logits, balance):
    return ol.gate(logits, gate.k, gate.score, balance, gate.n_groups, gate.topk_groups, gate.group_top, gate.renormalize,
                   gate.scale)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16", "fp8"])
def test_block_with_a_gate(dt, gather):
    from split_weight_expert_amd import MoEBlock
    name, kw = CASES[dt]
    if dt == "f32":
        kw = dict(kw, k=3)                             # two groups of two experts hold up to four
    cfg = shrink(synth.get_config(name), **kw)
    h = HostLayer(cfg)
    pl = [(0, e) if e < cfg.n_local else (1, e - cfg.n_local) for e in range(cfg.E)] + [(0, cfg.n_local)]
    store, table, x, wr, b = upload_layer(h, pl, [cfg.n_local + 1, cfg.E - cfg.n_local])
    gate = make_gate(cfg)
    balance = torch.randn(cfg.E, device=DEV) * 0.05
    balance[1] = -float("inf")                         # an expert out of service
    blk = MoEBlock(cfg.H, cfg.I, cfg.E, cfg.k, cfg.shared, cfg.dtype, DEV, gather=gather, gate=gate)
    bb = blk.forward(x, wr, b, table, balance_bias=balance)
    torch.cuda.synchronize()
    lg, gi = bb.logits.cpu().numpy(), bb.idx.cpu().numpy()
    oi, ow = oracle_gate(gate, lg, balance.cpu().numpy())
    np.testing.assert_array_equal(gi, oi)
    assert not (gi == 1).any()
    ref = omoe.moe_layer(to_np(x).astype(np.float32), h.wr, h.bias, cfg.k, lambda e: h.experts[e], lambda: h.shared,
                         precision=dt, routing=(lg, oi, ow))
    assert_close(to_np(bb.y), ref["y"], dt, f"block with a gate ({dt})")
    del store


def test_a_balance_bias_needs_a_gate():
    from split_weight_expert_amd import MoEBlock
    blk = MoEBlock(256, 128, 8, 2, 0, "f32", DEV)
    with pytest.raises(ValueError, match="needs a block with a gate"):
        blk.route(torch.zeros(4, 256, device=DEV), torch.zeros(8, 256, device=DEV), None, blk.buffers(4),
                  balance_bias=torch.zeros(8, device=DEV))
    with pytest.raises(ValueError, match="no normed input"):
        blk.forward_normed(torch.zeros(4, 256, device=DEV), None, None, None)


def test_a_forward_in_between_takes_the_normed_input():
    """forward() on the same buffers writes the codes that the norm wrote: no later layer may read the mixture."""
    from split_weight_expert_amd import MoEBlock
    name, kw = CASES["fp8"]
    cfg = shrink(synth.get_config(name), **kw)
    h = HostLayer(cfg)
    pl = [(0, e) if e < cfg.n_local else (1, e - cfg.n_local) for e in range(cfg.E)] + [(0, cfg.n_local)]
    store, table, x, wr, b = upload_layer(h, pl, [cfg.n_local + 1, cfg.E - cfg.n_local])
    blk = MoEBlock(cfg.H, cfg.I, cfg.E, cfg.k, cfg.shared, cfg.dtype, DEV, gate=make_gate(cfg))
    w = torch.ones(cfg.H, dtype=x.dtype, device=DEV)
    bb = blk.buffers(cfg.T)
    with pytest.raises(ValueError, match="shape"):
        blk.norm(x[1:], w, 1e-6, bb)
    with pytest.raises(ValueError, match="no normed input"):           # a refused norm is none
        blk.forward_normed(x, wr, b, table)
    blk.norm(x, w, 1e-6, bb)
    y0 = blk.forward_normed(x, wr, b, table, out=torch.empty_like(x)).x_norm.clone()
    first = bb.y_perm.clone()
    blk.forward_normed(x, wr, b, table, out=torch.empty_like(x))       # the input is still there
    assert torch.equal(bb.y_perm, first)
    blk.forward(x * 2, wr, b, table)
    with pytest.raises(ValueError, match="no normed input"):
        blk.forward_normed(x, wr, b, table)
    blk.norm(x, w, 1e-6, bb)
    blk.forward_normed(x, wr, b, table, out=torch.empty_like(x))
    torch.cuda.synchronize()
    assert torch.equal(bb.x_norm, y0) and torch.equal(bb.y_perm, first)
    del store


@pytest.mark.parametrize("dt,n_sets", [("f32", 2), ("bf16", 2), ("fp8", 2), ("bf16", 3)])
def test_pipeline_of_prenorm_layers(dt, n_sets):
    from split_weight_expert_amd import DWDPPipeline, api
    name, kw = CASES[dt]
    cfg = shrink(synth.get_config(name), **kw)
    host, layers, stores = build_layers(cfg)
    gate = make_gate(cfg)
    adt = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(4)
    for l, lw in enumerate(layers):
        lw.norm = (1 + 0.2 * torch.randn(cfg.H, generator=g)).to(DEV, adt)
        lw.norm_eps = 1e-6 * (l + 1)
        lw.balance_bias = (0.05 * torch.randn(cfg.E, generator=g)).to(DEV)
    L = len(layers)
    pipe = DWDPPipeline(cfg.H, cfg.I, cfg.E, cfg.k, cfg.shared, cfg.dtype, cfg.n_local, DEV, slot_sets=n_sets,
                        chunk_bytes=max(4096, stores[0].rec // 3 // 16 * 16), max_workgroups=3, gate=gate)
    x0 = torch.from_numpy(synth.tokens(cfg)).to(DEV, adt)
    fp8 = dt == "fp8"
    first = [torch.empty_like(x0), torch.empty(cfg.T, cfg.H, dtype=torch.uint8, device=DEV) if fp8 else None,
             torch.empty(cfg.T, cfg.H // 128, device=DEV) if fp8 else None]
    api.add_rmsnorm(x0, None, layers[0].norm, layers[0].norm_eps, None, *first)
    for call in range(2):
        outs = [torch.empty(cfg.T, cfg.H, dtype=adt, device=DEV) for _ in range(L)] if call == 0 else None
        seen = {}

        def after(l, b):
            seen[l] = (b.logits.clone(), b.idx.clone(), [None if t is None else t.clone()
                                                         for t in (b.x_norm, b.x_q, b.x_q_scale)])
        y = pipe.forward(x0, layers, outputs=outs, before_copy=lambda l: torch.cuda._sleep(SLEEP),
                         before_compute=lambda l: torch.cuda._sleep(SLEEP // 2), after_layer=after)
        torch.cuda.synchronize()
        if call == 1:                                  # the two alternating buffers give the same bits
            assert torch.equal(y, keep)
            break
        keep = y.clone()
        hcur = x0
        for l in range(L):
            xn, xq, xs = first if l == 0 else seen[l - 1][2]
            z = to_np(hcur).astype(np.float64)
            lw, hl = layers[l], host[l]
            # the sum that was normed is the unrounded one: half a step of the type from the stored one
            z_err = np.abs(z) * (U32 if dt == "f32" or l == 0 else 2.0 ** -8) * (0 if l == 0 else 1)
            check_norm(z, z_err, lw.norm.double().cpu().numpy(), lw.norm_eps, "f32" if dt == "f32" else "bf16", y=xn, q=xq,
                       q_scale=xs)
            lg, gi = seen[l][0].cpu().numpy(), seen[l][1].cpu().numpy()
            lr = omoe.router_logits(to_np(xn), to_np(lw.w_router), hl["b"])
            assert np.abs(lg - lr).max() <= 1e-5 * np.sqrt((lr ** 2).mean())
            oi, ow = oracle_gate(gate, lg, lw.balance_bias.cpu().numpy())
            np.testing.assert_array_equal(gi, oi, err_msg=f"layer {l} routing")
            tokens = omoe.dequant_groups(xq.cpu().numpy(), xs.cpu().numpy()) if fp8 else to_np(xn)
            ref = omoe.moe_layer(tokens.astype(np.float32), hl["wr"], hl["b"], cfg.k, lambda e, hl=hl: hl["experts"][e],
                                 lambda hl=hl: hl["shared"], precision=dt, routing=(lg, oi, ow))
            assert_close(to_np(outs[l]), z + ref["y"], dt, f"layer {l} ({dt})")
            hcur = outs[l]
    del stores
