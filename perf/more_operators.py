"""Further operators of the package's public API, as a user's program calls them.

  boundary  api.combine_branch_add_rmsnorm  the boundary between two layers whose blocks end in a norm of their own, a
                                            gate and a scale: weighted unpermute, norm, gate, scaled residual addition,
                                            and the next layer's norm
  branch    api.branch_add_rmsnorm          the same for a dense branch (an attention or dense FFN output)
  balance   api.balance_loss, api.gate_backward
                                            per-expert counts, the balance loss and the z loss of each sequence, and
                                            the logits' gradient of both losses and of the gate's weights
  experts   api.quantize_tokens_int8, api.moe_grouped_ffn_tokens
                                            the grouped SwiGLU expert FFN in 8-bit integers, with scales for each token
                                            and each weight channel

`run` computes them either with the package (`own`) or in their plain form: elementary torch operations in fp32,
rounded once at the end.  `exact` is the definition in fp64, written apart from the plain form.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    r1 = dict(H=7168, I=2048, k=8, shared=1)
    return [
        # the layer boundary of one token of one request
        dict(name="boundary-decode-1", op="boundary", T=1, H=7168, E=256, k=8, shared=1, dtype="bf16", norm=True,
             gate=False, token_gate=False, scale=1.0, residual_scale=1.0, fp8=False),
        # of a decode step of 64 requests, a gate for each channel and the next fp8 layer's codes
        dict(name="boundary-decode-64", op="boundary", T=64, H=7168, E=256, k=8, shared=1, dtype="bf16", norm=True,
             gate=True, token_gate=False, scale=1.0, residual_scale=1.0, fp8=True),
        # of an 8K-token prefill chunk, the branch scaled down and the next fp8 layer's codes
        dict(name="boundary-prefill-8k", op="boundary", T=8192, H=7168, E=256, k=8, shared=1, dtype="bf16", norm=True,
             gate=False, token_gate=False, scale=0.22, residual_scale=1.0, fp8=True),
        # the attention branch of a 16K-token prefill chunk: its norm, the residual addition, the block's norm
        dict(name="branch-prefill-16k", op="branch", T=16384, H=7168, dtype="bf16", norm=True, gate=False,
             token_gate=False, scale=1.0, residual_scale=1.0, fp8=False),
        # fp32, a width that no vector load divides, both gates, a scaled residual
        dict(name="branch-f32-odd", op="branch", T=1000, H=1001, dtype="f32", norm=True, gate=True, token_gate=True,
             scale=0.5, residual_scale=1.5, fp8=False),
        # a small micro-batch of one sequence
        dict(name="balance-64", op="balance", T=64, E=256, k=8, seqs=1, score="sigmoid", renorm=True, scale=2.5, pad=0),
        # a 16K-token batch of four sequences
        dict(name="balance-16k", op="balance", T=16384, E=256, k=8, seqs=4, score="sigmoid", renorm=True, scale=2.5,
             pad=0),
        # a softmax gate over an odd number of experts, many short sequences, padding behind the last
        dict(name="balance-ragged", op="balance", T=4097, E=60, k=6, seqs=33, score="softmax", renorm=False, scale=1.0,
             pad=101),
        # one token through int8 experts: its nine experts' weights are the work
        dict(name="experts-decode-1", op="experts", T=1, E=64, dtype="bf16", **r1),
        # a decode step of 64 requests
        dict(name="experts-decode-64", op="experts", T=64, E=64, dtype="bf16", **r1),
        # an 8K-token prefill chunk
        dict(name="experts-prefill-8k", op="experts", T=8192, E=128, dtype="bf16", **r1),
        # a smaller layer, a ragged batch, no shared expert
        dict(name="experts-ragged", op="experts", T=777, H=2048, I=768, E=60, k=6, shared=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["boundary", "branch", "balance", "experts"])
    if op == "balance":
        T = _log(rng, 1, 16384)
        E = _log(rng, 8, 384)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(12, E)), seqs=_log(rng, 1, 64),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 1.5, 2.5]), pad=rng.choice([0, 0, T // 5]))
    if op == "experts":
        E = _log(rng, 2, 64)
        return dict(op=op, T=_log(rng, 1, 4096), H=256 * _log(rng, 1, 28), I=128 * _log(rng, 1, 16), E=E,
                    k=rng.randint(1, min(8, E)), shared=rng.randint(0, 1), dtype="bf16")
    fp8 = rng.random() < 0.4
    dtype = "bf16" if fp8 or rng.random() < 0.7 else "f32"
    c = dict(op=op, dtype=dtype, norm=rng.random() < 0.8, gate=rng.random() < 0.5, token_gate=rng.random() < 0.3,
             scale=rng.choice([1.0, 0.22, 0.5]), residual_scale=rng.choice([1.0, 1.0, 1.5]), fp8=fp8)
    if op == "boundary":
        return dict(c, T=_log(rng, 1, 4096), H=128 * _log(rng, 1, 56), E=rng.choice([16, 60, 128, 256]),
                    k=rng.randint(1, 8), shared=rng.randint(0, 1))
    return dict(c, T=_log(rng, 1, 16384 if dtype == "bf16" else 4096),
                H=128 * _log(rng, 1, 56) if fp8 else _log(rng, 16, 7168))


# ------------------------------------------------------------------------------------------- inputs

def _permutation(T, k, E, g, drop=0.0):
    """Experts of every token, and the row of each assignment when rows are ordered by expert, token and slot."""
    experts = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].reshape(-1)
    order = experts.sort(stable=True).indices
    rank = torch.empty_like(experts)
    rank[order] = torch.arange(T * k, device="cuda")
    if drop:
        rank[torch.rand(T * k, generator=g, device="cuda") < drop] = -1
    return experts, order, rank


def _prepare_rows(s, c, g, randn):
    T, H, dt = c["T"], c["H"], TORCH[c["dtype"]]
    # a residual stream: a few channels in a hundred are an order of magnitude larger than the rest
    channel = torch.where(torch.rand(H, generator=g, device="cuda") < 0.02, 12.0, 1.0)
    s["residual"] = (randn(T, H) * channel).to(dt)
    s["weight"] = (1.0 + 0.2 * randn(H)).to(dt)
    s["eps"] = 1e-6
    s["norm"] = (1.0 + 0.2 * randn(H)).to(dt) if c["norm"] else None
    s["gate"] = (0.3 + 0.1 * randn(H)).to(dt) if c["gate"] else None
    s["token_gate"] = torch.sigmoid(randn(T)) if c["token_gate"] else None
    if c["op"] == "branch":
        s["x"] = (randn(T, H) * 0.5).to(dt)
        return
    k = c["k"]
    s["x"] = (randn(T * k + c["shared"] * T, H) * 0.3).to(dt)
    s["inv_perm"] = _permutation(T, k, c["E"], g, drop=0.002)[2].to(torch.int32).view(T, k)
    s["topk_w"] = torch.softmax(randn(T, k), 1)


def _prepare_balance(s, c, g, randn):
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    # some experts are more popular than others; the chosen are the k best after a small balance bias
    s["logits"] = randn(T, E) * 1.5 + randn(E) * 0.5
    s["idx"] = (s["logits"] + randn(E) * 0.1).topk(k, 1).indices.to(torch.int32)
    # sequences of random lengths, some of them empty, in front of the padding
    cuts = (torch.rand(S - 1, generator=g, device="cuda") * (T - c["pad"] + 1)).long().sort().values
    ends = torch.tensor([0, T - c["pad"]], device="cuda")
    s["seq_offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    s["d_w"] = randn(T, k) / T
    s["d_balance"] = torch.full((S,), 1.0 / S, device="cuda")
    s["d_z"] = torch.full((S,), 0.1 / S, device="cuda")


def _prepare_experts(s, c, g, randn):
    T, H, I, E, k, shared = c["T"], c["H"], c["I"], c["E"], c["k"], c["shared"]
    G = E + shared
    channel = torch.where(torch.rand(H, generator=g, device="cuda") < 0.02, 6.0, 1.0)
    s["x"] = (randn(T, H) * channel).to(torch.bfloat16)

    def codes(n, m):
        # weights of each channel drawn from a normal distribution whose largest value is some four deviations
        w = torch.empty(G, n, m, dtype=torch.int8, device="cuda")
        for e in range(G):
            w[e] = (randn(n, m) * 30.0).round_().clamp_(-127, 127)
        return w

    s["w13"], s["w2"] = codes(2 * I, H), codes(H, I)
    s["s13"] = (0.75 + 0.5 * torch.rand(G, 2 * I, generator=g, device="cuda")) / (30.0 * math.sqrt(H))
    s["s2"] = (0.75 + 0.5 * torch.rand(G, H, generator=g, device="cuda")) / (30.0 * math.sqrt(I))
    experts, order, _ = _permutation(T, k, E, g)
    count = torch.bincount(experts, minlength=E)
    groups = torch.cat([count, count.new_full((shared,), T)])
    s["offsets"] = torch.cat([groups.new_zeros(1), groups.cumsum(0)]).to(torch.int32)
    s["perm_src"] = torch.cat([order // k, torch.arange(T * shared, device="cuda")]).to(torch.int32)
    s["live"], s["most"] = count.nonzero()[:, 0], int(count.max())


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": c}
    make = {"boundary": _prepare_rows, "branch": _prepare_rows, "balance": _prepare_balance, "experts": _prepare_experts}
    make[c["op"]](s, c, g, randn)
    return s


# --------------------------------------------------------------------------------------- plain forms

def _plain_rows(s):
    c = s["case"]
    dt = TORCH[c["dtype"]]
    if c["op"] == "branch":
        u = s["x"].float()
    else:
        T, k = s["inv_perm"].shape
        rows = s["inv_perm"].long()
        wt = torch.where(rows >= 0, s["topk_w"], 0.0)
        u = (s["x"][rows.clamp(min=0)].float() * wt[:, :, None]).sum(1)
        if c["shared"]:
            u = u + s["x"][T * k:].float()
    if s["norm"] is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + s["eps"]) * s["norm"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    if s["token_gate"] is not None:
        u = u * s["token_gate"][:, None]
    total = s["residual"].float() * c["residual_scale"] + u * c["scale"]
    y = total * torch.rsqrt((total * total).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {"sum": total.to(dt), "y": y.to(dt)}
    if c["fp8"]:
        v = y.view(len(y), -1, 128)
        amax = v.abs().amax(2)
        scale = torch.where(amax == 0, 1.0, amax / 448.0)
        out["codes"] = (v / scale[:, :, None]).clamp(-448, 448).to(F8).view_as(y)
        out["scale"] = scale
    return out


def _plain_balance(s):
    c = s["case"]
    l, k, E = s["logits"], c["k"], c["E"]
    T = c["T"]
    idx = s["idx"].long()
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    soft = e / e.sum(1, keepdim=True)
    lse = (top + torch.log(e.sum(1, keepdim=True)))
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
        p = score / score.sum(1, keepdim=True)
        slope = 1.0 / (1.0 + torch.exp(l))           # 1 - score: a score's derivative by its logit over the score
    else:
        score, p, slope = soft, soft, torch.ones_like(soft)
    # which sequence holds a token, as rows of ones
    t, off = torch.arange(T, device=l.device), s["seq_offsets"]
    member = ((t >= off[:-1, None]) & (t < off[1:, None])).float()
    n = (off[1:] - off[:-1]).float()[:, None]
    inv = torch.where(n > 0, 1.0 / n, 0.0)
    hot = torch.zeros_like(l).scatter_add_(1, idx, torch.ones_like(idx, dtype=l.dtype))
    counts = member @ hot
    probs = member @ p * inv
    f = counts * inv * (E / k)
    out = {"counts": counts.to(torch.int32), "probs": probs, "balance": (f * probs).sum(1),
           "z": (member @ (lse * lse) * inv)[:, 0]}
    # gradients
    gb, gz = member.t() @ (s["d_balance"][:, None] * inv), member.t() @ (s["d_z"][:, None] * inv)
    ft = member.t() @ f
    d = gb * p * slope * (ft - (ft * p).sum(1, keepdim=True)) + gz * 2.0 * lse * soft
    chosen = score.gather(1, idx)
    if c["renorm"]:
        a = chosen / chosen.sum(1, keepdim=True)
        dw = c["scale"] * a * (s["d_w"] - (s["d_w"] * a).sum(1, keepdim=True)) * slope.gather(1, idx)
        d = d.scatter_add(1, idx, dw)
    else:
        dw = c["scale"] * s["d_w"] * chosen * slope.gather(1, idx)
        d = d.scatter_add(1, idx, dw)
        if c["score"] == "softmax":
            d = d - score * dw.sum(1, keepdim=True)
    out["d_logits"] = d
    return out


def _int8_rows(v):
    amax = v.abs().amax(-1, keepdim=True)
    scale = torch.where(amax == 0, 1.0, amax / 127.0)
    return torch.round(v / scale), scale


def _int8_ffn(xq, xs, w13, s13, w2, s2):
    """One SwiGLU FFN, or a batch of them."""
    h = (xq @ w13.float().transpose(-1, -2)) * xs * s13[..., None, :]
    g, u = h.chunk(2, -1)
    aq, sa = _int8_rows(g / (1.0 + torch.exp(-g)) * u)
    return (aq @ w2.float().transpose(-1, -2)) * sa * s2[..., None, :]


def _plain_experts(s):
    c = s["case"]
    T, E = c["T"], c["E"]
    routed = T * c["k"]
    xq, xs = _int8_rows(s["x"].float())
    y = torch.empty(len(s["perm_src"]) + 1, c["H"], device=xq.device)
    # the rows of every expert that has some in a block of its own, as high as the largest
    live, off = s["live"], s["offsets"].long()
    slot = torch.arange(s["most"], device=off.device)
    at = off[live, None] + slot
    src = s["perm_src"].long()[at.clamp(max=routed - 1)]
    block = _int8_ffn(xq[src], xs[src], s["w13"][live], s["s13"][live], s["w2"][live], s["s2"][live])
    at = torch.where(at < off[live + 1, None], at, len(y) - 1)       # the blocks' empty rows go behind the last
    y[at.view(-1)] = block.view(-1, c["H"])
    if c["shared"]:
        y[routed:-1] = _int8_ffn(xq, xs, s["w13"][E], s["s13"][E], s["w2"][E], s["s2"][E])
    return y[:-1].to(torch.bfloat16)


_PLAIN = {"boundary": _plain_rows, "branch": _plain_rows, "balance": _plain_balance, "experts": _plain_experts}


# --------------------------------------------------------------------------- the framework's operators

def _buffers(s):
    """What a program that calls the package keeps beside its inputs: outputs, workspaces, weights in their layout."""
    from split_weight_expert_amd import ExpertStore, api
    c = s["case"]
    T = c["T"]
    b = {"api": api}

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if c["op"] == "balance":
        S, E = c["seqs"], c["E"]
        b["gate"] = api.Gate(k=c["k"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        b["out"] = {"counts": empty(S, E, dtype=torch.int32), "probs": empty(S, E), "balance": empty(S), "z": empty(S),
                    "d_logits": empty(T, E)}
        b["ws"] = empty(api.balance_loss_workspace_bytes(T, E, S), dtype=torch.uint8)
    elif c["op"] == "experts":
        H, I, G = c["H"], c["I"], c["E"] + c["shared"]
        rows = len(s["perm_src"])
        store = ExpertStore(H, I, api.INT8, [G])
        for e in range(G):
            store.load_int8(0, e, s["w13"][e], s["s13"][e], s["w2"][e], s["s2"][e])
        b["store"], b["table"] = store, store.table([(0, e) for e in range(G)])
        b["x_q"], b["x_scale"] = empty(T, H, dtype=torch.int8), empty(T)
        b["y"] = empty(rows, H, dtype=torch.bfloat16)
        b["ws"] = empty(api.workspace_bytes(api.OP_GROUPED_FFN, T, c["k"], c["E"], H, I, api.INT8, c["shared"]),
                        dtype=torch.uint8)
    else:
        dt = TORCH[c["dtype"]]
        b["branch"] = api.Branch(norm=s["norm"], eps=s["eps"], gate=s["gate"], scale=c["scale"],
                                 residual_scale=c["residual_scale"])
        b["out"] = {"sum": empty(T, c["H"], dtype=dt), "y": empty(T, c["H"], dtype=dt)}
        b["q"] = b["q_scale"] = None
        if c["fp8"]:
            b["q"], b["q_scale"] = empty(T, c["H"], dtype=torch.uint8), empty(T, c["H"] // 128)
            b["out"]["codes"], b["out"]["scale"] = b["q"].view(F8), b["q_scale"]
    return b


def _own(s):
    b = s.get("own")
    if b is None:
        b = s["own"] = _buffers(s)
    c, api = s["case"], b["api"]
    op = c["op"]
    if op == "balance":
        out = b["out"]
        api.balance_loss(s["logits"], s["idx"], b["gate"], out["counts"], out["probs"], out["balance"], out["z"],
                         b["ws"], seq_offsets=s["seq_offsets"])
        api.gate_backward(s["logits"], s["idx"], b["gate"], out["d_logits"], d_w=s["d_w"], counts=out["counts"],
                          d_balance=s["d_balance"], d_z=s["d_z"], seq_offsets=s["seq_offsets"])
        return out
    if op == "experts":
        api.quantize_tokens_int8(s["x"], b["x_q"], b["x_scale"])
        api.moe_grouped_ffn_tokens(0, b["table"], c["E"] + c["shared"], s["offsets"], s["perm_src"], b["x_q"],
                                   b["x_scale"], c["H"], c["I"], api.INT8, b["y"], b["ws"])
        return b["y"]
    out = b["out"]
    if op == "branch":
        api.branch_add_rmsnorm(s["x"], s["residual"], b["branch"], s["weight"], s["eps"], sum_out=out["sum"], y=out["y"],
                               q=b["q"], q_scale=b["q_scale"], token_gate=s["token_gate"])
    else:
        api.combine_branch_add_rmsnorm(s["x"], s["inv_perm"], s["topk_w"], c["shared"], s["residual"], b["branch"],
                                       s["weight"], s["eps"], sum_out=out["sum"], y=out["y"], q=b["q"],
                                       q_scale=b["q_scale"], token_gate=s["token_gate"])
    return out


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ the work

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "balance":
        S, E, k = c["seqs"], c["E"], c["k"]
        # the gradient needs the counts of a whole sequence, so both passes read the logits and the choice
        n = 2 * (T * E * 4 + T * k * 4 + (S + 1) * 4) + T * k * 4 + T * E * 4 + S * E * 12 + S * 16
        return {"bytes": n, "flops": 25 * T * E}
    if c["op"] == "experts":
        H, I, E, shared = c["H"], c["I"], c["E"], c["shared"]
        rows = T * c["k"] + shared * T
        touched = E * (1 - (1 - c["k"] / E) ** T) + shared
        n = touched * (3 * H * I + 4 * (2 * I + H)) + T * H * 2 + rows * (4 + H * 2)
        return {"bytes": int(n), "flops": 6 * H * I * rows}
    H, e = c["H"], TORCH[c["dtype"]].itemsize
    n = 3 * T * H * e + H * e * (1 + c["norm"] + c["gate"]) + 4 * T * c["token_gate"]
    n += T * H + T * (H // 128) * 4 if c["fp8"] else 0
    if c["op"] == "branch":
        return {"bytes": n + T * H * e, "flops": 10 * T * H}
    src = c["k"] + c["shared"]
    return {"bytes": n + T * H * e * src + T * c["k"] * 8, "flops": (2 * src + 10) * T * H}


# ----------------------------------------------------------------- the definition in 64 bits, by itself

def _exact_rows(s):
    c = s["case"]
    H = c["H"]
    if c["op"] == "branch":
        u = s["x"].double()
    else:
        T, k = s["inv_perm"].shape
        u = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            r = s["inv_perm"][:, j].long()
            live = r >= 0
            u[live] += s["x"][r[live]].double() * s["topk_w"][live, j, None].double()
        if c["shared"]:
            u += s["x"][T * k:]
    if c["norm"]:
        u = s["norm"].double() * u / (u.square().sum(1) / H + s["eps"]).sqrt()[:, None]
    u *= c["scale"]
    if c["gate"]:
        u *= s["gate"].double()
    if c["token_gate"]:
        u *= s["token_gate"].double()[:, None]
    z = u.add_(s["residual"].double(), alpha=c["residual_scale"])
    y = s["weight"].double() * z / (z.square().sum(1) / H + s["eps"]).sqrt()[:, None]
    out = {"sum": z, "y": y}
    if c["fp8"]:
        v = y.reshape(-1, 128)
        scale = v.abs().max(1).values / 448
        scale[scale == 0] = 1.0
        v = v / scale[:, None]
        # E4M3 has 3 fraction bits and its smallest normal exponent is -6: round to its spacing, ties to even
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out["codes"] = ((v / step).round() * step).view_as(y)
        out["scale"] = scale.view(len(y), -1)
    return out


def _exact_balance(s):
    """The losses as they are written, sequence by sequence, and their gradient by differentiation."""
    c = s["case"]
    k, E, S = c["k"], c["E"], c["seqs"]
    l = s["logits"].double().requires_grad_(True)
    score = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    p = score / score.sum(1, keepdim=True)
    z2 = torch.logsumexp(l, 1).square()
    idx = s["idx"].long()
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    off = s["seq_offsets"].tolist()
    none = torch.zeros((), dtype=torch.float64, device="cuda")
    balance, z, probs = [], [], []
    for a, b in zip(off[:-1], off[1:]):
        if a == b:
            balance.append(none)
            z.append(none)
            probs.append(none.expand(E))
            continue
        f = torch.bincount(idx[a:b].reshape(-1), minlength=E).double() * E / (k * (b - a))
        probs.append(p[a:b].mean(0))
        balance.append((f * probs[-1]).sum())
        z.append(z2[a:b].mean())
    balance, z = torch.stack(balance), torch.stack(z)
    total = (balance * s["d_balance"]).sum() + (z * s["d_z"]).sum() + (c["scale"] * w * s["d_w"]).sum()
    total.backward()
    return {"counts": None, "probs": torch.stack(probs).detach(), "balance": balance.detach(), "z": z.detach(),
            "d_logits": l.grad}


def _exact_experts(s):
    c = s["case"]
    I = c["I"]

    def to_int8(v):
        scale = v.abs().max(1, keepdim=True).values / 127
        scale[scale == 0] = 1.0
        return (v / scale).round(), scale

    q, qs = to_int8(s["x"].double())
    off = s["offsets"].tolist()
    y = torch.empty(len(s["perm_src"]), c["H"], dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a == b:
            continue
        src = s["perm_src"][a:b].long()
        h = (q[src] @ s["w13"][e].double().t()) * (qs[src] * s["s13"][e].double())
        act, sa = to_int8(h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:])
        y[a:b] = (act @ s["w2"][e].double().t()) * (sa * s["s2"][e].double())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"boundary": _exact_rows, "branch": _exact_rows, "balance": _exact_balance, "experts": _exact_experts}[
        case["op"]](s)
