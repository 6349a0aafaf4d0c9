"""The operators in a run of layers as a program uses them: int8 layers with branches in a block and in the pipeline, and
the router's losses and gradient of a routed batch."""
import numpy as np
import pytest
import torch

from oracle import balance as ob

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, H, I, E, k = 70, 512, 256, 8, 2


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_weight_expert_amd import api
    return api


def layers(api, n, dtype, seed=0):
    from split_weight_expert_amd import ExpertStore
    from split_weight_expert_amd.moe import DTYPES
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g).to(DEV)
    out = []
    for _ in range(n):
        st = ExpertStore(H, I, DTYPES[dtype], [E + 1])
        for e in range(E + 1):
            st.load(0, e, r(I, H) / H ** 0.5, r(I, H) / H ** 0.5, r(H, I) / I ** 0.5)
        out.append(dict(store=st, table=st.table([(0, e) for e in range(E + 1)]), wr=(r(E, H) / H ** 0.5).bfloat16(),
                        bb=r(E) * 0.05, norm=(1 + 0.1 * r(H)).bfloat16(),
                        branch=api.Branch(norm=(1 + 0.1 * r(H)).bfloat16(), gate=0.5 + 0.1 * r(H), scale=0.8, residual_scale=1.1)))
    return out


GATE = dict(k=k, score="sigmoid", n_groups=4, topk_groups=2, group_top=2, scale=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "int8"])
def test_a_stack_of_layers_with_branches(api, dtype):
    """forward_normed layer by layer gives the bits of the single calls: norm with codes, route, FFN on them, boundary."""
    from split_weight_expert_amd import MoEBlock
    gate = api.Gate(**GATE)
    ls = layers(api, 3, dtype)
    block, parts = MoEBlock(H, I, E, k, 1, dtype, gate=gate), MoEBlock(H, I, E, k, 1, dtype, gate=gate)
    attn, h0 = ((torch.randn(T, H, generator=torch.Generator().manual_seed(i)) * (i + 1)).bfloat16().to(DEV) for i in range(2))
    tg = torch.rand(T, generator=torch.Generator().manual_seed(3)).to(DEV)
    # the block's input is the norm of an attention branch added to the stream
    b = block.buffers(T)
    h = torch.empty_like(h0)
    block.norm(attn, ls[0]["norm"], 1e-6, b, residual=h0, sum_out=h, branch=ls[0]["branch"], token_gate=tg)
    want, x = torch.empty_like(h0), torch.empty_like(h0)
    q, qs = (None if t is None else torch.empty_like(t) for t in (b.x_q, b.x_q_scale))
    api.branch_add_rmsnorm(attn, h0, ls[0]["branch"], ls[0]["norm"], 1e-6, sum_out=want, y=x, q=q, q_scale=qs, token_gate=tg)
    assert torch.equal(h, want)
    for n, l in enumerate(ls):
        nxt = ls[n + 1]["norm"] if n + 1 < len(ls) else None
        assert torch.equal(x, b.x_norm)
        p = parts.buffers(T)
        parts.route(x, l["wr"], None, p, balance_bias=l["bb"])
        parts.permute(x, p)
        if q is not None:                    # the codes of the unrounded norm in the place of those of x
            p.x_q.copy_(q)
            p.x_q_scale.copy_(qs)
        parts.ffn(l["table"], p)
        hin = h.clone()
        block.forward_normed(h, l["wr"], None, l["table"], nxt, 1e-6, out=h, balance_bias=l["bb"], branch=l["branch"], token_gate=tg)
        assert torch.equal(p.idx, b.idx) and torch.equal(p.w, b.w) and torch.equal(p.y_perm, b.y_perm)
        want = torch.empty_like(h)
        outs = {} if nxt is None else dict(y=x, q=q, q_scale=qs)
        api.combine_branch_add_rmsnorm(p.y_perm, p.inv_perm, p.w, 1, hin, l["branch"], nxt, 1e-6, sum_out=want, token_gate=tg, **outs)
        assert torch.equal(h, want)
    with pytest.raises(ValueError, match="no normed input"):
        block.forward_normed(h, ls[0]["wr"], None, ls[0]["table"])


def test_an_unnamed_sum_needs_its_handle(api):
    """A norm of a branch whose sum went nowhere is of no tensor: its handle is needed."""
    from split_weight_expert_amd import MoEBlock
    l = layers(api, 1, "int8")[0]
    block = MoEBlock(H, I, E, k, 1, "int8", gate=api.Gate(**GATE))
    x = torch.randn(T, H, device=DEV).bfloat16()
    b = block.buffers(T)
    handle = block.norm(x, l["norm"], 1e-6, b, branch=l["branch"])
    with pytest.raises(ValueError, match="no normed input of this h"):
        block.forward_normed(x, l["wr"], None, l["table"])
    block.forward_normed(x, l["wr"], None, l["table"], normed=handle)
    block.norm(x, l["norm"], 1e-6, b)
    block.forward_normed(x, l["wr"], None, l["table"])


def test_pipeline_of_int8_layers_with_branches(api):
    """DWDPPipeline over int8 layers with branches: the bits of the same layers run one by one."""
    from split_weight_expert_amd import DWDPPipeline, LayerWeights, MoEBlock
    n_local = 3
    gate = api.Gate(**GATE)
    ls = layers(api, 3, "int8", seed=5)
    pipe = DWDPPipeline(H, I, E, k, 1, "int8", n_local, gate=gate, chunk_bytes=1 << 16)
    weights = []
    for l in ls:
        st = l["store"]
        rec = st.buffers[0].view(E + 1, st.rec)
        resident = torch.cat([rec[:n_local].reshape(-1), rec[E]])
        peers = rec[n_local:E].reshape(-1).clone()
        l["keep"] = peers
        weights.append(LayerWeights(l["wr"], None, resident, [(peers.data_ptr(), 0, peers.numel())], balance_bias=l["bb"],
                                    norm=l["norm"], branch=l["branch"]))
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).bfloat16().to(DEV)
    block = MoEBlock(H, I, E, k, 1, "int8", gate=gate)
    h = x.clone()
    block.norm(h, ls[0]["norm"], 1e-6, block.buffers(T))
    for n, l in enumerate(ls):
        nxt = ls[n + 1]["norm"] if n + 1 < len(ls) else None
        block.forward_normed(h, l["wr"], None, l["table"], nxt, 1e-6, out=h, balance_bias=l["bb"], branch=l["branch"])
    for _ in range(2):
        assert torch.equal(pipe.forward(x, weights), h)


@pytest.mark.parametrize("gated", [False, True])
def test_router_losses_of_a_routed_batch(api, gated):
    from split_weight_expert_amd import MoEBlock
    gate = api.Gate(**GATE) if gated else None
    l = layers(api, 1, "bf16")[0]
    block = MoEBlock(H, I, E, k, 1, "bf16", gate=gate)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).bfloat16().to(DEV)
    b = block.buffers(T)
    block.route(x, l["wr"], None, b, balance_bias=l["bb"] if gated else None)
    off = torch.tensor([0, 20, 20, 65], dtype=torch.int32, device=DEV)
    r = block.balance(b, off)
    score, scale = ("sigmoid", 2.0) if gated else ("softmax", 1.0)
    want = ob.losses(b.logits.cpu().numpy(), b.idx.cpu().numpy(), score, off.tolist())
    assert np.array_equal(r.counts.cpu().numpy(), want[0]) and r.counts.sum().item() == 65 * k
    # |logits| is a few units: (2.2 * 10 + 12) 2^-23 and the sums' roundings
    for got, w in zip((r.probs, r.balance, r.z), want[1:]):
        assert np.allclose(got.cpu().numpy(), w, rtol=1e-5, atol=0)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).to(DEV)
    db, dz = torch.tensor([1.0, 2.0, -1.0], device=DEV), torch.tensor([0.1, 0.2, 0.3], device=DEV)
    d = block.gate_backward(b, dw, r, db, dz)
    ref, size = ob.backward(b.logits.cpu().numpy(), b.idx.cpu().numpy(), score, True, scale, off.tolist(),
                            *(t.double().cpu().numpy() for t in (dw, db, dz)))
    assert (np.abs(d.double().cpu().numpy() - ref) <= 1e-5 * size + 1e-36).all()
    # a whole batch, and the weights alone, on another stream
    one = block.balance(b)
    assert one.counts.shape == (1, E) and one.counts.sum().item() == T * k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(T, E, device=DEV)
    torch.cuda.synchronize()
    block.gate_backward(b, dw, out=out, stream=side)
    again = block.balance(b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again.counts, one.counts) and torch.equal(again.balance, one.balance)
    ref, size = ob.backward(b.logits.cpu().numpy(), b.idx.cpu().numpy(), score, True, scale, None, dw.double().cpu().numpy())
    assert (np.abs(out.double().cpu().numpy() - ref) <= 1e-5 * size + 1e-36).all()


def test_training_step_of_a_router_in_a_graph(api):
    """Gate, losses and gradient captured and replayed with new logits; every replay against the eager result."""
    Tn, En, kn = 300, 48, 4
    gate = api.Gate(k=kn, score="sigmoid")
    l = torch.empty(Tn, En, device=DEV)
    off = torch.tensor([0, 100, 290], dtype=torch.int32, device=DEV)
    idx, w = torch.empty(Tn, kn, dtype=torch.int32, device=DEV), torch.empty(Tn, kn, device=DEV)
    o = [torch.empty(2, En, dtype=torch.int32, device=DEV), torch.empty(2, En, device=DEV), torch.empty(2, device=DEV),
         torch.empty(2, device=DEV)]
    ws = torch.empty(api.balance_loss_workspace_bytes(Tn, En, 2), dtype=torch.uint8, device=DEV)
    dw, db, dz, d = torch.randn(Tn, kn, device=DEV), torch.ones(2, device=DEV), torch.ones(2, device=DEV), torch.empty_like(l)

    def step():
        api.gate_topk(l, gate, idx, w)
        api.balance_loss(l, idx, gate, *o, ws=ws, seq_offsets=off)
        api.gate_backward(l, idx, gate, d, dw, o[0], db, dz, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        l.normal_()
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = [*o, d, w, idx]
    for i in range(4):
        l.copy_(torch.randn(Tn, En, generator=torch.Generator().manual_seed(i)))
        step()
        want = [t.clone() for t in outs]
        torch.cuda.synchronize()
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, v) for t, v in zip(outs, want))
