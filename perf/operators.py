"""Measured cases of the operators of a drafted tree's verification forward.

Three operators, used one after the other in a speculative decoding step:

* ``tree_qkv_rope``      -- RMS norm of the query and key heads, the rotation at
  each node's own position, and the write of the keys and values to the tree's
  places in the cache;
* ``tree_attention``     -- attention of every tree node over a prefix shared
  by the whole batch, its sequence's own cached positions, and its ancestors
  in the tree;
* ``verify_tree_sample`` -- sampling verification of the tree: a walk from the
  root that draws each next token from the target's distribution with a given
  uniform number and goes on while a child holds the token drawn.

``run`` computes them with elementary torch operations (``own`` false) or with
this repository's kernels (``own`` true).
"""
import math

import numpy as np
import torch

own = False

MAX_CHILDREN = 4   # children per tree node, as the tree workload's trees
BOOSTED = 8        # likely tokens of a target row
STEP = 0.7         # distance of their logits (at temperature 1)
LIFT = 1.7         # the first one's logit above the log-sum of the rest
ROWS_VISITED = 2.5  # mean rows of a sequence that a walk reads, for these trees and rows


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one stream at low latency: a 60-node tree over a 128k vocabulary
        dict(name="sample_one_stream", op="sample", B=1, N=60, V=128256, depth=6, T=1.0, dtype="bf16"),
        # the tree workload of the benchmark
        dict(name="sample_tree_batch", op="sample", B=16, N=60, V=128256, depth=6, T=1.0, dtype="bf16"),
        # rows of an odd length, which start at no vector boundary
        dict(name="sample_odd_vocabulary", op="sample", B=7, N=23, V=32003, depth=4, T=0.75, dtype="bf16"),
        # a serving batch with float32 logits and the largest vocabulary
        dict(name="sample_large_f32", op="sample", B=64, N=32, V=151936, depth=8, T=0.625, dtype="f32"),
        # a short chat turn with a small chain of drafts, heads not shared
        dict(name="attention_short_chain", op="attention", B=1, N=5, Hkv=8, G=1, D=64, ctx=300, P=0, chain=True),
        # plain decoding: one token of every sequence
        dict(name="attention_decode", op="attention", B=64, N=1, Hkv=8, G=4, D=128, ctx=4096, P=0, chain=True),
        # the tree workload behind a few thousand cached tokens
        dict(name="attention_tree", op="attention", B=16, N=60, Hkv=8, G=4, D=128, ctx=4096, P=0, chain=False),
        # a long document: few sequences, one long axis to split
        dict(name="attention_long", op="attention", B=3, N=33, Hkv=8, G=5, D=128, ctx=65536, P=0, chain=False),
        # a system prompt that the whole batch shares
        dict(name="attention_shared_prefix", op="attention", B=64, N=16, Hkv=8, G=4, D=128, ctx=700, P=8192, chain=False),
        # one stream
        dict(name="qkv_one_stream", op="qkv", B=1, N=60, Hkv=8, G=4, D=128, ctx=4096, rot=128, norm=True, interleaved=False),
        # odd sizes: a chain of 7, half of each head rotated, pairs side by side
        dict(name="qkv_partial_interleaved", op="qkv", B=37, N=7, Hkv=3, G=5, D=64, ctx=1000, rot=32, norm=False, interleaved=True),
        # a serving batch of trees
        dict(name="qkv_large", op="qkv", B=128, N=60, Hkv=8, G=4, D=128, ctx=2048, rot=128, norm=True, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "attention", "qkv"])
    if op == "sample":
        V = _log_int(rng, 500, 151936)
        if rng.random() < 0.5:
            V = max(8, V // 8 * 8)
        N = _log_int(rng, 1, 64)
        return dict(op=op, B=min(_log_int(rng, 1, 64), max(1, 300_000_000 // (N * V))), N=N, V=V, depth=rng.randint(1, 8),
                    T=rng.randint(16, 40) / 32, dtype=rng.choice(["bf16", "f32"]))
    G, Hkv, D = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    B, N = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
    if op == "attention":
        P = 0 if rng.random() < 0.5 else _log_int(rng, 1, 16384)
        ctx = _log_int(rng, 1, 65536)
        most = 300_000_000 // (B * N * G * Hkv)  # scores of one query head and node
        P = min(P, max(1, most // 2)) if P else 0
        ctx = max(1, min(ctx, most - P, 3_000_000 // (B * Hkv)))
        return dict(op=op, B=B, N=N, Hkv=Hkv, G=G, D=D, ctx=ctx, P=P, chain=rng.random() < 0.3)
    norm = rng.random() < 0.6
    return dict(op=op, B=B, N=N, Hkv=Hkv, G=G, D=D, ctx=_log_int(rng, 1, 4096), rot=rng.choice([D, D, D // 2, 0, 6]),
                norm=norm, interleaved=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _trees(rng, B, N, depth, chain):
    """Parents, depths and ancestor relation of B trees of N nodes."""
    par = np.full((B, N), -1, np.int32)
    dep = np.zeros((B, N), np.int32)
    kids = np.zeros((B, N), np.int32)
    anc = np.zeros((B, N, N), bool)
    rows = np.arange(B)
    anc[:, 0, 0] = True
    for v in range(1, N):
        if chain:
            p = np.full(B, v - 1)
        else:
            key = rng.random((B, v))
            key[kids[:, :v] >= MAX_CHILDREN] -= 1.0  # only where every place is taken
            key[dep[:, :v] >= depth] -= 2.0          # never: the root is always less deep
            p = key.argmax(axis=1)
        par[:, v] = p
        dep[:, v] = dep[rows, p] + 1
        kids[rows, p] += 1
        anc[:, v] = anc[rows, p]
        anc[:, v, v] = True
    return par, dep, anc


def _pack(anc):
    """Ancestor relation as words of 32 bits, bit u % 32 of word u / 32."""
    B, N, _ = anc.shape
    W = (N + 31) // 32
    full = np.zeros((B, N, W * 32), np.uint8)
    full[:, :, :N] = anc
    return np.packbits(full, axis=2, bitorder="little").view(np.uint32).view(np.int32).reshape(B, N, W).copy()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, dtype=dtype, **dev)

    def cuda(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    B, N = case["B"], case["N"]
    s = dict(case=dict(case))
    if case["op"] == "sample":
        V, T = case["V"], case["T"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        par, dep, _ = _trees(rng, B, N, case["depth"], False)
        # every row: a wide background and BOOSTED likely tokens, which the children hold in turn
        logits = normal(B, N, V, dtype=dt).mul_(2.0 * T)
        likely = torch.randint(0, V, (B, N, BOOSTED), generator=gen, **dev)
        lift = T * (math.log(V) + 2.0 + LIFT - STEP * torch.arange(BOOSTED, **dev))
        logits.scatter_(2, likely, lift.to(dt).expand(B, N, BOOSTED).contiguous())
        rank = np.zeros((B, N), np.int64)
        seen = np.zeros((B, N), np.int64)
        rows = np.arange(B)
        for v in range(1, N):
            rank[:, v] = seen[rows, par[:, v]]
            seen[rows, par[:, v]] += 1
        tokens = likely[torch.arange(B, **dev)[:, None], cuda(np.maximum(par, 0)).long(), cuda(rank % BOOSTED)].int()
        tokens[:, 0] = -1
        s.update(logits=logits, tokens=tokens.contiguous(), parents=cuda(par),
                 u=torch.rand(B, case["depth"] + 1, generator=gen, **dev))
        return s
    Hkv, G, D, ctx = case["Hkv"], case["G"], case["D"], case["ctx"]
    # own lengths between half of ctx and ctx, the root among them
    base = rng.integers(max(1, ctx // 2), ctx + 1, size=B).astype(np.int32)
    L = ctx + N
    par, dep, anc = _trees(rng, B, N, 8, case.get("chain", False))
    s.update(base=cuda(base))
    if case["op"] == "attention":
        s.update(q=normal(B, N, Hkv * G, D), k=normal(B, L, Hkv, D), v=normal(B, L, Hkv, D), scale=1.0 / math.sqrt(D),
                 mask=None if case["chain"] else cuda(_pack(anc)), pk=None, pv=None)
        if case["P"]:
            s.update(pk=normal(case["P"], Hkv, D), pv=normal(case["P"], Hkv, D))
        return s
    H = Hkv * (G + 2)
    s.update(qkv=normal(B, N, H, D), depth=cuda(dep), eps=1e-6, rot=case["rot"],
             qw=1 + 0.1 * normal(D) if case["norm"] else None, kw=1 + 0.1 * normal(D) if case["norm"] else None,
             inv_freq=(500000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, **dev) / max(1, case["rot"]))).float(),
             offset=1000, k=torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, **dev),
             v=torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, **dev))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"sample": _own_sample, "attention": _own_attention, "qkv": _own_qkv}[op](state)
    return {"sample": _plain_sample, "attention": _plain_attention, "qkv": _plain_qkv}[op](state)


def _own_sample(s):
    import speculative_decoding_verification_56_gb300 as sv
    c = s["case"]
    if "ws" not in s:  # kept by a decoding loop, with the outputs
        B, W = c["B"], c["depth"] + 1
        code = sv.SPEC_DTYPE_BF16 if c["dtype"] == "bf16" else sv.SPEC_DTYPE_F32
        s["ws"] = sv.alloc_workspace(sv.SPEC_MODE_TREE_SAMPLE, B, c["N"], c["V"], code)
        s["out"] = (torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, W, dtype=torch.int32, device="cuda"),
                    torch.empty(B, W, dtype=torch.int32, device="cuda"), torch.empty(B, W, dtype=torch.float32, device="cuda"))
    n, path, toks, probs = s["out"]
    sv.spec_verify_tree_sample(s["logits"], s["tokens"], s["parents"], s["u"], c["T"], c["depth"], n, path, toks, probs, s["ws"])
    return dict(accepted_len=n, path_nodes=path, out_tokens=toks, out_probs=probs)


def _own_attention(s):
    import speculative_decoding_verification_56_gb300 as sv
    q = s["q"]
    if "ws" not in s:
        s["ws"] = sv.alloc_tree_attention_workspace(q, s["k"], s["pk"])
        s["out"] = (torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device="cuda"))
    out, lse = s["out"]
    sv.spec_tree_attention(q, s["k"], s["v"], s["mask"], s["base"], s["scale"], out, lse, s["ws"], prefix_k=s["pk"], prefix_v=s["pv"])
    return dict(out=out, lse=lse)


def _own_qkv(s):
    import speculative_decoding_verification_56_gb300 as sv
    if "ws" not in s:
        B, N, _, D = s["qkv"].shape
        s["ws"] = sv.alloc_workspace(sv.SPEC_MODE_TREE_QKV, B, N, 1, sv.SPEC_DTYPE_BF16)
        s["out"] = torch.empty(B, N, s["case"]["Hkv"] * s["case"]["G"], D, dtype=torch.bfloat16, device="cuda")
    sv.spec_tree_qkv_rope(s["qkv"], s["qw"], s["kw"], s["eps"], s["inv_freq"], s["base"], s["depth"], s["out"], s["k"], s["v"], s["ws"],
                          pos_offset=s["offset"], interleaved=s["case"]["interleaved"])
    return dict(q=s["out"], k=s["k"], v=s["v"])


def _plain_sample(s):
    """Every node's token drawn at once (64 bits: a draw next to a border must
    fall on its side), then the walk as products of the matching edges."""
    c = s["case"]
    B, N, V, W = c["B"], c["N"], c["V"], c["depth"] + 1
    par, tok = s["parents"].long(), s["tokens"].long()
    node = torch.arange(N, device="cuda")
    # ancestors: the closure of the parent relation, by repeated squaring
    up = (par[:, :, None] == node) & (node[:, None] > 0)
    reach = (up | torch.eye(N, dtype=torch.bool, device="cuda")).float()
    for _ in range(4):  # paths of up to 16 edges
        reach = (reach @ reach).clamp_(max=1)
    depth = reach.sum(2).long() - 1
    e = s["logits"].double() / c["T"]
    e = (e - e.amax(2, keepdim=True)).exp_()
    total = e.sum(2)
    cum = e.cumsum(2)
    u = s["u"].double().gather(1, depth.clamp(max=W - 1))
    x = (cum <= (u * total)[:, :, None]).sum(2).clamp_(max=V - 1)
    p = e.gather(2, x[:, :, None])[:, :, 0] / total
    # an edge is taken if the child holds the parent's token, and no sibling before it does
    hit = (tok == x.gather(1, par.clamp(min=0))) & (node > 0)
    twin = (par[:, :, None] == par[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & (node < node[:, None])
    step = (hit & ~(twin & hit[:, None, :]).any(2) & (depth < W)) | (node == 0)
    on = (reach * ~step[:, None, :]).sum(2) == 0
    n = (on.sum(1) - 1).int()
    at = torch.where(on, depth, W)
    path = torch.full((B, W + 1), -1, dtype=torch.long, device="cuda").scatter_(1, at.clamp(max=W), node.expand(B, N))[:, :W]
    used = path >= 0
    out = torch.where(used, x.gather(1, path.clamp(min=0)), -1)
    probs = torch.where(used, p.gather(1, path.clamp(min=0)), 0)
    return dict(accepted_len=n, path_nodes=path.int(), out_tokens=out.int(), out_probs=probs.float())


def _visible(s, L):
    """[B, N, L]: which own positions each node sees."""
    B, N = s["case"]["B"], s["case"]["N"]
    node = torch.arange(N, device="cuda")
    if s["mask"] is None:
        tree = (node[None, :] <= node[:, None]).expand(B, N, N)
    else:
        tree = (s["mask"].long()[:, :, node // 32] >> (node % 32)) & 1 != 0
    root = s["base"].long()[:, None] - 1
    rel = torch.arange(L, device="cuda") - root
    inside = (rel >= 0) & (rel < N)
    seen = tree.gather(2, rel.clamp(0, N - 1)[:, None, :].expand(B, N, L))
    return (rel < 0)[:, None, :] | (inside[:, None, :] & seen)


def _plain_attention(s):
    c = s["case"]
    B, N, Hkv, G, D = (c[k] for k in ("B", "N", "Hkv", "G", "D"))
    L = s["k"].shape[1]
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) * s["scale"]
    z = q @ s["k"].float().permute(0, 2, 3, 1)
    z = z.view(B, Hkv, N, G, L).masked_fill_(~_visible(s, L)[:, None, :, None, :], -math.inf).view(B, Hkv, N * G, L)
    m = z.amax(3, keepdim=True)
    if s["pk"] is not None:
        zp = torch.einsum("bhrd,phd->bhrp", q, s["pk"].float())
        m = torch.maximum(m, zp.amax(3, keepdim=True))
    e = (z - m).exp_()
    total = e.sum(3, keepdim=True)
    o = e @ s["v"].float().permute(0, 2, 1, 3)
    if s["pk"] is not None:
        e = (zp - m).exp_()
        total = total + e.sum(3, keepdim=True)
        o = o + torch.einsum("bhrp,phd->bhrd", e, s["pv"].float())
    out = (o / total).view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, D)
    lse = (m + total.log()).view(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, Hkv * G)
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _plain_qkv(s):
    c = s["case"]
    B, N, Hkv, G, D, rot = (c[k] for k in ("B", "N", "Hkv", "G", "D", "rot"))
    Hq = Hkv * G
    x = s["qkv"].float()
    qk, v = x[:, :, : Hq + Hkv], s["qkv"][:, :, Hq + Hkv:]
    if s["qw"] is not None:
        qk = qk * torch.rsqrt(qk.square().mean(3, keepdim=True) + s["eps"])
        qk = torch.cat([qk[:, :, :Hq] * s["qw"].float(), qk[:, :, Hq:] * s["kw"].float()], 2)
    pos = s["offset"] + s["base"].double()[:, None] - 1 + s["depth"].double()
    angle = pos[:, :, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(3)
    else:
        a, b = qk[..., : rot // 2], qk[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(torch.bfloat16)
    at = s["base"].long()[:, None] - 1 + torch.arange(N, device="cuda")
    rows = torch.arange(B, device="cuda")[:, None]
    s["k"][rows, at] = qk[:, :, Hq:]
    s["v"][rows, at] = v
    return dict(q=qk[:, :, :Hq].contiguous(), k=s["k"], v=s["v"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    B, N = case["B"], case["N"]
    if case["op"] == "sample":
        rows = B * min(ROWS_VISITED, case["depth"] + 1, N)  # the rows that the walks come to
        size = 2 if case["dtype"] == "bf16" else 4
        W = case["depth"] + 1
        return dict(bytes=rows * case["V"] * size + B * (8 * N + 4 * W) + B * (4 + 12 * W), flops=rows * case["V"] * 4)
    Hkv, G, D = case["Hkv"], case["G"], case["D"]
    Hq = Hkv * G
    if case["op"] == "attention":
        own_len = B * 0.75 * case["ctx"]
        seen = N * (own_len + B * case["P"]) + B * N * min(N, 5)
        W = 0 if case["chain"] else (N + 31) // 32
        moved = (own_len + B * N + case["P"]) * Hkv * D * 4 + B * N * (Hq * D * 4 + Hq * 4 + 4 * W) + 4 * B
        return dict(bytes=moved, flops=4 * seen * Hq * D)
    return dict(bytes=B * N * (Hq + 2 * Hkv) * D * 4 + B * (4 + 4 * N), flops=B * N * (Hq + Hkv) * D * 8)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"sample": _exact_sample, "attention": _exact_attention, "qkv": _exact_qkv}[case["op"]](case, s)


def _exact_sample(c, s):
    B, N, W = c["B"], c["N"], c["depth"] + 1
    par, tok, u = s["parents"].tolist(), s["tokens"].tolist(), s["u"].tolist()
    n = np.zeros(B, np.int32)
    path, out = np.full((B, W), -1, np.int32), np.full((B, W), -1, np.int32)
    probs = np.zeros((B, W))
    for b in range(B):
        cur = 0
        for d in range(W):
            p = torch.softmax(s["logits"][b, cur].double() / c["T"], 0)
            x = int(torch.searchsorted(p.cumsum(0), u[b][d], right=True))
            x = min(x, c["V"] - 1)
            path[b, d], out[b, d], probs[b, d], n[b] = cur, x, float(p[x]), d
            cur = next((v for v in range(1, N) if par[b][v] == cur and tok[b][v] == x), None)
            if cur is None:
                break
    return dict(accepted_len=n, path_nodes=path, out_tokens=out, out_probs=probs)


def _exact_attention(c, s):
    B, N, Hkv, G, D = (c[k] for k in ("B", "N", "Hkv", "G", "D"))
    out = torch.empty(B, N, Hkv * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, N, Hkv * G, dtype=torch.float64, device="cuda")
    bits = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        root = int(s["base"][b]) - 1
        sees = np.tril(np.ones((N, N), bool)) if bits is None else np.array(
            [[bits[b, v, w // 32] >> (w % 32) & 1 for w in range(N)] for v in range(N)], bool)
        sees = torch.from_numpy(sees).cuda()
        for h in range(Hkv):
            k, v = s["k"][b, : root + N, h].double(), s["v"][b, : root + N, h].double()
            hidden = torch.zeros(N, root + N, dtype=torch.bool, device="cuda")
            hidden[:, root:] = ~sees
            if s["pk"] is not None:
                k, v = torch.cat([s["pk"][:, h].double(), k]), torch.cat([s["pv"][:, h].double(), v])
                hidden = torch.cat([torch.zeros(N, c["P"], dtype=torch.bool, device="cuda"), hidden], 1)
            for g in range(G):
                z = s["q"][b, :, h * G + g].double() @ k.T * s["scale"]
                z[hidden] = -math.inf
                lse[b, :, h * G + g] = torch.logsumexp(z, 1)
                out[b, :, h * G + g] = torch.softmax(z, 1) @ v
    return dict(out=out, lse=lse)


def _exact_qkv(c, s):
    Hkv, G, D, rot, N = (c[k] for k in ("Hkv", "G", "D", "rot", "N"))
    Hq = Hkv * G
    x = s["qkv"].double()
    q, k, v = x[:, :, :Hq], x[:, :, Hq: Hq + Hkv], x[:, :, Hq + Hkv:]
    if s["qw"] is not None:
        q = q / (q.pow(2).sum(3, keepdim=True) / D + s["eps"]).sqrt() * s["qw"].double()
        k = k / (k.pow(2).sum(3, keepdim=True) / D + s["eps"]).sqrt() * s["kw"].double()
    at = s["base"].double()[:, None] - 1 + s["depth"].double() + s["offset"]

    def turn(y):
        y = y.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            z = torch.polar(torch.ones_like(at), at * s["inv_freq"][i].double())[:, :, None] * torch.complex(y[..., a], y[..., b])
            y[..., a], y[..., b] = z.real, z.imag
        return y

    q, k = turn(q), turn(k)
    kc, vc = s["k"].double(), s["v"].double()
    for b, r in enumerate(s["base"].tolist()):
        kc[b, r - 1: r - 1 + N], vc[b, r - 1: r - 1 + N] = k[b], v[b]
    return dict(q=q, k=kc, v=vc)
