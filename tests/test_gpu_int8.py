"""int8 experts on the GPU: the row quantiser and the packed weights exactly, the grouped FFN against fp64.

Tolerances.  Integer sums are exact, so a pre-activation has three roundings (the sum's conversion and two scales):
3 2^-24 of its value.  silu(g) u: its exponential's relative error is (1.1 |g| + 2) 2^-23, the reciprocal's 2^-23, and a
relative error e of g moves silu(g) by at most (1 + |g|) e; together (3.5 |g| + 12) 2^-23 of |A|.  A code of A is
the rounding of a value that far from the exact one, so |code scale - A| is at most half a step more.  y from the GPU's own codes
of A has three roundings in fp32 and one to bf16, half a step: 2^-8 (1 + 2^-10)."""
import numpy as np
import pytest
import torch

from oracle import int8 as o8

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from split_weight_expert_amd import api
    return api


QUANT = [(1, 8), (5, 64), (7, 128), (9, 136), (300, 256), (3, 512), (70, 520), (17, 2048), (4, 7168), (2049, 1000), (3, 16384),
         (2, 20000), (2, 32768), (2, 40008)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", QUANT)
def test_quantiser_is_exact(api, rows, cols, dt):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 20)
    x[0, 0] = 0
    if rows > 4:
        x[1] = 0
        x[2, 3] = float("nan")
        x[3, cols - 1] = float("-inf")
        x[4] = 1e-39
    x = x.to(dt).to(DEV)
    q = torch.full((rows + 1, cols), 99, dtype=torch.int8, device=DEV)
    s = torch.full((rows + 1,), 7.0, device=DEV)
    api.quantize_tokens_int8(x, q[:rows], s[:rows])
    want, ws = o8.rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(q[:rows].cpu().numpy(), want)
    np.testing.assert_array_equal(s[:rows].cpu().numpy(), ws)
    assert (q[rows:] == 99).all() and (s[rows:] == 7).all()


def test_quantiser_divides_as_ieee_does(api):
    """Values at and beside every tie: (2 m + 1) / 2 scales, one ulp to both sides, for scales of every kind."""
    g = np.random.default_rng(0)
    amax = np.concatenate([np.exp(g.normal(size=200) * 30), [127.0, 254.0, 1.0, 2.0 ** 100, 3.3e38, 1e-30]]).astype(np.float32)
    amax = np.minimum(amax, np.float32(3.3e38))
    s = np.maximum(amax / np.float32(127), np.float32(2.0 ** -126))
    ties = (np.arange(-127, 127) + 0.5).astype(np.float32)
    with np.errstate(over="ignore"):
        mid = (s[:, None].astype(np.float64) * ties).astype(np.float32)
    x = np.concatenate([amax[:, None], np.nextafter(mid, np.float32(-np.inf)), mid, np.nextafter(mid, np.float32(np.inf)),
                        np.zeros((len(s), 5), np.float32)], 1)
    x = np.clip(x, -amax[:, None], amax[:, None])
    assert x.shape[1] % 8 == 0
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    sc = torch.empty(len(x), device=DEV)
    api.quantize_weight_int8(torch.from_numpy(x).to(DEV), q, sc)
    want, ws = o8.rows(x)
    np.testing.assert_array_equal(sc.cpu().numpy(), ws)
    np.testing.assert_array_equal(q.cpu().numpy(), want)


def test_packed_layout(api):
    N, K = 96, 384
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, generator=torch.Generator().manual_seed(1)).to(DEV)
    out = torch.empty(N * K, dtype=torch.int8, device=DEV)
    api.pack_weights(w, out, api.INT8)
    # 1 KB blocks (row block, column block): lane l holds row l % 32, columns 16 (l // 32) .. + 15
    want = w.view(N // 32, 32, K // 32, 2, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    assert torch.equal(out, want)


class Layer:
    """G groups of int8 weights with rows per group, and the GPU's results for them."""

    def __init__(self, api, rows, H, I, seed, T=None, extreme=False):
        from split_weight_expert_amd import ExpertStore
        g = torch.Generator().manual_seed(seed)
        G, n = len(rows), sum(rows)
        T = max(1, n // 2) if T is None else T
        self.api, self.H, self.I, self.G, self.n, self.T = api, H, I, G, n, T

        def codes(*s):
            return torch.full(s, -128, dtype=torch.int8) if extreme else (torch.randn(*s, generator=g) * 40).round().clamp(-128, 127).to(torch.int8)
        self.w13, self.w2 = codes(G, 2 * I, H), codes(G, H, I)
        self.s13 = (0.5 + torch.rand(G, 2 * I, generator=g)) / (40 * H ** 0.5)
        self.s2 = (0.5 + torch.rand(G, H, generator=g)) / (40 * I ** 0.5)
        self.x = (torch.randn(T, H, generator=g) * 2).bfloat16()
        self.src = torch.randint(0, T, (n,), generator=g, dtype=torch.int32)
        self.off = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
        self.store = ExpertStore(H, I, api.INT8, [G // 2, G - G // 2])
        place = [(0, e) if e < G // 2 else (1, e - G // 2) for e in range(G)]
        for e, (b, s) in enumerate(place):
            self.store.load_int8(b, s, self.w13[e].to(DEV), self.s13[e].to(DEV), self.w2[e].to(DEV), self.s2[e].to(DEV))
        self.table = self.store.table(place)
        self.q, self.qs = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        api.quantize_tokens_int8(self.x.to(DEV), self.q, self.qs)
        if extreme:
            self.q.fill_(-128)
        need = api.workspace_bytes(api.OP_GROUPED_FFN, n, 1, G, H, I, api.INT8, 0)
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
        self.srcd, self.offd = self.src.to(DEV), self.off.to(DEV)
        self.y = torch.full((n + 1, H), 7.0, dtype=torch.bfloat16, device=DEV)

    def run(self, stage=0):
        self.api.moe_grouped_ffn_tokens(stage, self.table, self.G, self.offd, self.srcd, self.q, self.qs, self.H, self.I,
                                        self.api.INT8, self.y[:self.n], self.ws)
        return self.y[:self.n]

    def a(self):
        """A's codes and scales as the workspace holds them."""
        n, I = self.n, self.I
        o = (n * I + 255) // 256 * 256
        return self.ws[:n * I].view(torch.int8).view(n, I).cpu().numpy(), self.ws[o:o + 4 * n].view(torch.float32).cpu().numpy()

    def check(self, groups=None):
        self.run()
        assert (self.y[self.n:] == 7).all()
        a, sa = self.a()
        y = self.y[:self.n].double().cpu().numpy()
        q, qs = self.q.cpu().numpy(), self.qs.cpu().numpy()
        flips = 0
        for e in range(self.G) if groups is None else groups:
            r = slice(int(self.off[e]), int(self.off[e + 1]))
            if r.start == r.stop:
                continue
            src = self.src[r].numpy()
            A, gate = o8.gate_up(q[src], qs[src], self.w13[e].numpy(), self.s13[e].numpy())
            dA = np.abs(A) * (3.5 * np.abs(gate) + 12) * 2 * U
            amax, dmax = np.abs(A).max(1), dA.max(1)
            s = sa[r].astype(np.float64)
            assert (np.abs(s - amax / 127) <= dmax / 127 + 4 * U * amax / 127).all()
            # the window's own 2^-15 steps: a code of 127 times the quotient's rounding
            assert (np.abs(a[r] * s[:, None] - A) <= s[:, None] * (0.5 + 2.0 ** -15) + dA).all()
            want = o8.product(a[r], sa[r], self.w2[e].numpy(), self.s2[e].numpy())
            assert (np.abs(y[r] - want) <= np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -10) + 1e-38).all()
            flips += (a[r] != np.rint(A / (amax / 127)[:, None])).mean()
        return flips


# rows per group: empty groups, single rows, tails of every 32-row block, and every tile height
ROWS = [([1], 256, 128), ([0, 3, 0, 1, 33, 0], 256, 128), ([31, 32, 33, 64, 65, 1, 0, 20], 512, 256),
        ([50, 90, 1, 63, 64, 129], 768, 128), ([100, 200, 0, 161, 97, 128], 256, 384), ([300, 0, 257, 511, 33, 224, 700], 512, 256),
        ([5, 3, 2, 0, 8, 1, 1, 9], 7168, 2048), ([260, 190, 250], 2304, 640), ([2000], 256, 128), ([64, 40, 0, 100], 256, 1152),
        # tiles of 128 rows: 512 of them with groups of 64 or more, 256 with groups of more than 128
        ([64, 65, 127, 128, 0, 63, 100, 70] * 4, 256, 2048), ([129, 255, 300, 31, 161, 96, 0, 330] * 2, 512, 1024)]


@pytest.mark.parametrize("rows,H,I", ROWS)
def test_grouped_ffn(api, rows, H, I):
    Layer(api, rows, H, I, len(rows) + H).check()


def test_largest_sums(api):
    """Codes of -128 on both sides over the widest K of this test: sums of 2^14 K, whole numbers past fp32's."""
    L = Layer(api, [40, 7], 8192, 128, 5, extreme=True)
    L.run(1)
    a32 = L.a()
    q, qs = L.q.cpu().numpy(), L.qs.cpu().numpy()
    for e in range(2):
        r = slice(int(L.off[e]), int(L.off[e + 1]))
        src = L.src[r].numpy()
        A, gate = o8.gate_up(q[src], qs[src], L.w13[e].numpy(), L.s13[e].numpy())
        amax = np.abs(A).max(1)
        dmax = (np.abs(A) * (3.5 * np.abs(gate) + 12) * 2 * U).max(1)
        assert (np.abs(a32[1][r] - amax / 127) <= dmax / 127 + 4 * U * amax / 127).all()


def test_stages_static_workspace_and_permuted_rows_agree(api):
    """Stage 1 then 2, the library's own workspace, and rows already permuted: the same bits."""
    L = Layer(api, [30, 0, 70, 129, 5], 512, 256, 3)
    want = L.run().clone()
    L.y.fill_(0)
    L.run(1)
    L.run(2)
    assert torch.equal(L.y[:L.n], want)
    y = torch.empty_like(want)
    api.moe_grouped_ffn_tokens_static(0, L.table, L.G, L.offd, L.srcd, L.q, L.qs, L.H, L.I, api.INT8, y)
    assert torch.equal(y, want)
    y.zero_()
    src = L.srcd.long()
    api.moe_grouped_ffn(L.table, L.G, L.offd, L.q[src].contiguous(), L.qs[src].contiguous(), L.H, L.I, api.INT8, y, L.ws)
    assert torch.equal(y, want)


def test_a_nan_token_stays_in_its_rows(api):
    L = Layer(api, [33, 40, 64], 256, 128, 8)
    clean = L.run().clone()
    x = L.x.clone()
    x[3, 100] = float("nan")
    x[7, 0] = float("inf")
    api.quantize_tokens_int8(x.to(DEV), L.q, L.qs)
    y = L.run()
    bad = ((L.srcd == 3) | (L.srcd == 7))
    assert bad.any() and torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


def test_indices_out_of_range_are_clamped(api):
    L = Layer(api, [20, 20], 256, 128, 9)
    L.srcd[3], L.srcd[30] = -5, 1 << 30
    y = L.run().clone()
    L.srcd[3], L.srcd[30] = 0, L.T - 1
    assert torch.equal(L.run(), y)


@pytest.mark.parametrize("shared", [0, 1])
def test_block_and_store_from_masters(api, shared):
    """ExpertStore.load quantises fp32 masters by output channel; the block's result is near the layer in fp64."""
    from split_weight_expert_amd import ExpertStore, MoEBlock
    T, H, I, E, k = 100, 512, 256, 8, 2
    g = torch.Generator().manual_seed(4)
    ws = [[torch.randn(*s, generator=g) / s[1] ** 0.5 for s in ((I, H), (I, H), (H, I))] for _ in range(E + shared)]
    st = ExpertStore(H, I, api.INT8, [E + shared])
    for e, w in enumerate(ws):
        st.load(0, e, *(t.to(DEV) for t in w))
        q13, s13 = o8.rows(torch.cat(w[:2]).numpy())
        assert np.array_equal(st.views(0, e)[2].cpu().numpy(), s13)
    x, wr = torch.randn(T, H, generator=g).bfloat16().to(DEV), (torch.randn(E, H, generator=g) / H ** 0.5).bfloat16().to(DEV)
    block = MoEBlock(H, I, E, k, shared, "int8")
    b = block.forward(x, wr, None, st.table([(0, e) for e in range(E + shared)]))
    xq, xs = o8.rows(x.float().cpu().numpy())
    idx, w = b.idx.cpu().numpy(), b.w.double().cpu().numpy()
    want = np.zeros((T, H))
    size = np.zeros((T, H))
    for e in range(E + shared):
        q13, s13 = o8.rows(torch.cat(ws[e][:2]).numpy())
        q2, s2 = o8.rows(ws[e][2].numpy())
        A, gate = o8.gate_up(xq, xs, q13, s13)
        a, sa = o8.rows(A)
        y = o8.product(a, sa, q2, s2)
        # a code may land beside the oracle's where A is next to a tie: one step of A through the channel's weights
        step = sa[:, None].astype(np.float64) * np.abs(q2.astype(np.float64) * s2[:, None]).max(1)
        f = np.ones(T) if e == E else (w * (idx == e)).sum(1)
        want += f[:, None] * y
        size += f[:, None] * (np.abs(y) * 2.0 ** -8 * 1.01 + 2 * step)
    got = b.y.double().cpu().numpy()
    assert (np.abs(got - want) <= size + np.abs(want) * 2.0 ** -8).all()


def test_graph_replays(api):
    """Quantiser and FFN captured into a graph, replayed with new tokens between eager runs."""
    L = Layer(api, [30, 64, 3, 200], 512, 256, 13)
    x = L.x.to(DEV)

    def step():
        api.quantize_tokens_int8(x, L.q, L.qs)
        L.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_((torch.randn(L.T, L.H, generator=torch.Generator().manual_seed(i)) * (i + 1)).bfloat16())
        step()
        want = L.y.clone()
        torch.cuda.synchronize()
        L.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.y[:L.n], want[:L.n])


def test_no_rows(api):
    y = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(0, 256, dtype=torch.int8, device=DEV)
    api.moe_grouped_ffn_tokens(0, None, 3, torch.zeros(4, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV),
                               q, torch.empty(0, device=DEV), 256, 128, api.INT8, y, None)
    api.quantize_tokens_int8(q.bfloat16(), q, torch.empty(0, device=DEV))
