"""Pre-norm layers of MoEBlock on the GPU, whose buffers all batches of one size share."""
import pytest
import torch

import synth
from synth.configs import shrink
from tests.gpu_util import HostLayer, need_gpu, upload_layer
from tests.test_gpu_layer_block import CASES, DEV, make_gate

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
