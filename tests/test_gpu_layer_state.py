"""Pre-norm layers of MoEBlock on the GPU, whose buffers all batches of one size share, and in gather mode."""
import numpy as np
import pytest
import torch

import synth
from oracle import moe as omoe
from synth.configs import shrink
from tests.gpu_util import HostLayer, assert_close, need_gpu, to_np, upload_layer
from tests.test_gpu_layer import U32, check_norm
from tests.test_gpu_layer_block import CASES, DEV, make_gate, oracle_gate

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def layer(dt, gather=False):
    from split_weight_expert_amd import MoEBlock
    name, kw = CASES[dt]
    if dt == "f32":
        kw = dict(kw, k=3)                             # two groups of two experts hold up to four
    cfg = shrink(synth.get_config(name), **kw)
    h = HostLayer(cfg)
    pl = [(0, e) if e < cfg.n_local else (1, e - cfg.n_local) for e in range(cfg.E)] + [(0, cfg.n_local)]
    store, table, x, wr, b = upload_layer(h, pl, [cfg.n_local + 1, cfg.E - cfg.n_local])
    blk = MoEBlock(cfg.H, cfg.I, cfg.E, cfg.k, cfg.shared, cfg.dtype, DEV, gather=gather, gate=make_gate(cfg))
    return cfg, h, blk, store, table, x, wr, b


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16", "fp8"])
def test_batches_of_one_size_do_not_mix(dt, gather):
    cfg, _, blk, store, table, x, wr, b = layer(dt, gather)
    w = torch.ones(cfg.H, dtype=x.dtype, device=DEV)
    other = (x.flip(0) * 0.5).contiguous()
    want = {}
    for n, t in (("x", x), ("other", other)):
        blk.norm(t, w, 1e-6, blk.buffers(cfg.T))
        want[n] = torch.empty_like(t)
        blk.forward_normed(t, wr, b, table, out=want[n])
    bb = blk.buffers(cfg.T)
    blk.norm(x, w, 1e-6, bb)
    blk.norm(other, w, 1e-6, bb)
    out = torch.zeros_like(x)
    with pytest.raises(ValueError, match="no normed input of this h"):
        blk.forward_normed(x, wr, b, table, out=out)
    torch.cuda.synchronize()
    assert not out.any()
    blk.forward_normed(other, wr, b, table, out=out)
    assert torch.equal(out, want["other"])
    with pytest.raises(ValueError, match="no normed input of this h"):
        blk.forward_normed(x, wr, b, table, out=out)
    blk.norm(x, w, 1e-6, bb)
    blk.forward_normed(x, wr, b, table, out=out)
    assert torch.equal(out, want["x"])
    del store


def test_the_first_norm_on_a_side_stream():
    """x_norm's memory is not one that the current stream, far behind, still reads from a tensor freed on it."""
    from split_weight_expert_amd import MoEBlock
    T, H = 512, 2048
    blk = MoEBlock(H, 256, 8, 2, 0, "bf16", DEV)
    bb = blk.buffers(T)
    x, w = torch.ones(T, H, dtype=torch.bfloat16, device=DEV), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    old, keep = torch.full_like(x, 3), torch.zeros_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    keep.copy_(old)
    del old                                            # reads it only after the sleep
    blk.norm(x, w, 0.0, bb, stream=side)
    torch.cuda.synchronize()
    assert (keep == 3).all() and (bb.x_norm == 1).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "fp8"])
def test_two_prenorm_layers_in_gather_mode(dt):
    """Both layers of a pair against the oracle on the GPU's own input of that layer; the second one's norm comes from
    the first one's boundary.  Codes of fp8 rows are the token quantiser's of the normed rows."""
    from split_weight_expert_amd import api
    cfg, hl, blk, store, table, x, wr, b = layer(dt, gather=True)
    g = torch.Generator().manual_seed(3)
    w = [(1 + 0.2 * torch.randn(cfg.H, generator=g)).to(DEV, x.dtype) for _ in range(2)]
    bb = blk.buffers(cfg.T)
    h = [x, torch.empty_like(x), torch.empty_like(x)]
    blk.norm(x, w[0], 1e-6, bb)
    for l in range(2):
        xn = bb.x_norm.clone()
        z = to_np(h[l]).astype(np.float64)
        # the boundary normed the unrounded sum: half a step of the type from the stored one
        z_err = np.abs(z) * (0 if l == 0 else U32 if dt == "f32" else 2.0 ** -8)
        check_norm(z, z_err, w[l].double().cpu().numpy(), 1e-6, "f32" if dt == "f32" else "bf16", y=xn)
        blk.forward_normed(h[l], wr, b, table, next_weight=w[1] if l == 0 else None, out=h[l + 1])
        torch.cuda.synchronize()
        lg = bb.logits.cpu().numpy()
        oi, ow = oracle_gate(blk.gate, lg, None)
        np.testing.assert_array_equal(bb.idx.cpu().numpy(), oi)
        if dt == "fp8":
            q, s = torch.empty(cfg.T, cfg.H, dtype=torch.uint8, device=DEV), torch.empty(cfg.T, cfg.H // 128, device=DEV)
            api.quantize_tokens_fp8(xn, q, s)
            src = bb.perm_src.long()
            assert torch.equal(bb.x_perm, q[src]) and torch.equal(bb.x_perm_scale, s[src])
        ref = omoe.moe_layer(to_np(xn).astype(np.float32), hl.wr, hl.bias, cfg.k, lambda e: hl.experts[e], lambda: hl.shared,
                             precision=dt, routing=(lg, oi, ow))
        assert_close(to_np(h[l + 1]), z + ref["y"], dt, f"layer {l} ({dt}, gather)")
    del store


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_both_modes_of_a_normed_layer_give_the_same_bits(dt):
    outs = []
    for gather in (False, True):
        cfg, _, blk, store, table, x, wr, b = layer(dt, gather)
        blk.norm(x, torch.ones(cfg.H, dtype=x.dtype, device=DEV), 1e-6, blk.buffers(cfg.T))
        out = torch.empty_like(x)
        blk.forward_normed(x, wr, b, table, out=out)
        torch.cuda.synchronize()
        outs.append(out)
        del store
    assert torch.equal(*outs)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_normed_layer_without_a_gate(dt, gather):
    """The plain top-k's block inside a residual layer is forward() on the normed rows, and the residual: the boundary adds
    it in fp32 and rounds once, forward() rounds its own sum first."""
    from split_weight_expert_amd import MoEBlock
    cfg, _, _, store, table, x, wr, b = layer(dt, gather)
    blk = MoEBlock(cfg.H, cfg.I, cfg.E, cfg.k, cfg.shared, cfg.dtype, DEV, gather=gather)
    blk.norm(x, torch.ones(cfg.H, dtype=x.dtype, device=DEV), 1e-6, blk.buffers(cfg.T))
    out = torch.empty_like(x)
    bb = blk.forward_normed(x, wr, b, table, out=out)
    idx, xn = bb.idx.clone(), bb.x_norm.clone()
    y = torch.empty_like(x)
    blk.forward(xn, wr, b, table, out=y)
    torch.cuda.synchronize()
    assert torch.equal(idx, bb.idx)
    u = 2.0 ** -8 if dt == "bf16" else U32
    want = x.double() + y.double()
    # y's rounding, the fp32 addition, the output's rounding
    assert ((out.double() - want).abs() <= u * y.double().abs() + (u + U32) * (1 + u) * (want.abs() + u * y.double().abs())).all()
    del store
