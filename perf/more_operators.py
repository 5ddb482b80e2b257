"""Measured cases of the operators around a 4-bit key-value cache in pages.

* ``attention`` -- ``tree_attention_kv4``: attention of every tree node over its
  sequence's committed positions, held in 4 bits in pages, and its ancestors,
  still in bf16;
* ``store``     -- ``kv4_commit_path`` and ``kv4_read``: the accepted path's keys
  and values into the pages of every layer, and the pages back to bf16;
* ``fork``      -- ``kv_pages_fork``: every new sequence takes the pages of its
  parent (shared, the unfinished one copied where another writes it) and fresh
  pages to grow into; pages that nobody holds any more are free;
* ``compact``   -- ``kv_pages_compact``: the pages in use move to the lowest places;
* ``beam``      -- ``beam_select``: the best continuations over beams and vocabulary,
  whose parents are what the fork takes.

``run`` computes them with elementary torch operations (``own`` false) or with
this repository's kernels (``own`` true).
"""
import math

import numpy as np
import torch

own = False

MAX_CHILDREN = 4   # children per tree node, as the tree workload's trees
BLOCK = 16         # channels that share a scale
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the 4-bit codes


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a short chat turn with a small chain of drafts, heads not shared
        dict(name="attention_short_chain", op="attention", B=1, N=5, Hkv=8, G=1, D=64, ctx=300, page=16, chain=True),
        # plain decoding: one token of every sequence
        dict(name="attention_decode", op="attention", B=64, N=1, Hkv=8, G=4, D=128, ctx=4096, page=64, chain=True),
        # the benchmark's trees behind a few thousand committed tokens
        dict(name="attention_tree", op="attention", B=16, N=60, Hkv=8, G=4, D=128, ctx=4096, page=64, chain=False),
        # a long document: few sequences, one long axis to split
        dict(name="attention_long", op="attention", B=3, N=33, Hkv=8, G=5, D=128, ctx=65536, page=128, chain=False),
        # the step after a walk: a few accepted nodes of each tree, all layers, short sequences
        dict(name="store_paths", op="store", B=16, N=60, Hkv=8, D=128, ctx=150, page=16, layers=4, path=True),
        # prompts: every position of a chunk is stored, and handed over in bf16
        dict(name="store_prompts", op="store", B=5, N=1000, Hkv=8, D=128, ctx=500, page=64, layers=8, path=False),
        # four beams of one stream
        dict(name="fork_one_stream", op="fork", B=4, B2=4, ctx=300, grow=1, page=16, planes=4, Hkv=8, D=64, spare=16),
        # eight beams of each of eight requests, over the layers of a target
        dict(name="fork_batch", op="fork", B=64, B2=64, ctx=1000, grow=60, page=64, planes=32, Hkv=8, D=128, spare=200),
        # holes that finished requests left
        dict(name="compact_batch", op="compact", B=24, ctx=1500, page=64, planes=32, Hkv=8, D=128, spare=300),
        dict(name="compact_small", op="compact", B=3, ctx=200, page=32, planes=2, Hkv=3, D=64, spare=9),
        # four beams over a 128k vocabulary at low latency
        dict(name="beam_one_stream", op="beam", B=1, K=4, M=4, V=128256, T=1.0, dtype="bf16"),
        # a batch of requests with eight beams each: the largest logits
        dict(name="beam_batch", op="beam", B=64, K=8, M=8, V=128256, T=1.0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "store", "fork", "compact", "beam", "beam"])
    Hkv, D, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "attention":
        G = rng.choice([1, 2, 3, 4, 5, 8])
        B, N = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, 65536)
        ctx = max(1, min(ctx, 300_000_000 // (B * N * G * Hkv), 2_400_000 // (B * Hkv)))
        return dict(op=op, B=B, N=N, Hkv=Hkv, G=G, D=D, ctx=ctx, page=page, chain=rng.random() < 0.4)
    if op == "store":
        path = rng.random() < 0.5
        B, layers = _log_int(rng, 1, 32), _log_int(rng, 1, 8)
        N = _log_int(rng, 1, 64) if path else _log_int(rng, 1, 2048)
        most = 60_000 // (B * layers)  # positions of a sequence
        N = max(1, min(N, most // 2))
        return dict(op=op, B=B, N=N, Hkv=Hkv, D=D, ctx=max(1, min(_log_int(rng, 1, 1000), most - N)), page=page,
                    layers=layers, path=path)
    if op in ("fork", "compact"):
        B, planes = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
        ctx = _log_int(rng, 1, 2000)
        c = dict(op=op, B=B, ctx=ctx, page=page, planes=planes, Hkv=Hkv, D=D, spare=_log_int(rng, 4, 300))
        most = 1_600_000_000 // (planes * Hkv * D * 9 // 8)  # positions of the pool
        c["ctx"] = max(1, min(ctx, most // (4 * B) - 2 * page)) if most // (4 * B) > 2 * page else 1
        if op == "fork":
            c.update(B2=max(1, min(B, _log_int(rng, 1, 64))), grow=_log_int(rng, 1, 64))
        return c
    V = _log_int(rng, 500, 151936)
    if rng.random() < 0.5:
        V = max(16, V // 8 * 8)
    K = rng.randint(1, 12)
    return dict(op=op, B=max(1, min(_log_int(rng, 1, 64), 60_000_000 // (K * V))), K=K, M=rng.choice([K, rng.randint(1, 16)]),
                V=V, T=rng.randint(16, 40) / 32, dtype=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# the pages' format: of one head, 16 positions after 16 positions, codes of the
# keys [16, D / 2], their scales [16, D / 16], codes of the values, their scales
# ---------------------------------------------------------------------------

def _block_bytes(case):
    return case["page"] * case["D"] * 9 // 8


def _parts(pages, page, D):
    """Views of the pages' four parts, [..., heads, page / 16, 16, bytes]."""
    out, at = [], 0
    pages = pages.unflatten(-1, (page // 16, 18 * D))
    for width in (D // 2, D // BLOCK) * 2:
        out.append(pages[..., at: at + 16 * width].unflatten(-1, (16, width)))
        at += 16 * width
    return out


def _encode(x, e):
    """Codes (two channels to a byte) and scales of x float32 [..., D] with the
    exponents e, which broadcast against [..., 1, 1]."""
    y = x.unflatten(-1, (-1, BLOCK))
    unit = torch.exp2(e.float())
    s = (y.abs().amax(-1, keepdim=True) / 6 / unit).clamp(max=448).to(torch.float8_e4m3fn)
    step = s.float() * unit
    m = y.abs() / torch.where(step > 0, step, torch.inf)
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)).byte()
    code = (code + 8 * (y < 0)).byte().flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1).view(torch.uint8)


def _decode(codes, scales, e):
    """The values, float32 [..., D]."""
    table = torch.tensor(CODES + tuple(-c for c in CODES), device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * torch.exp2(e.float())
    return (table[pair].unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


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

    op, B = case["op"], case["B"]
    s = dict(case=dict(case))
    if op == "beam":
        K, V, T = case["K"], case["V"], case["T"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        logits = normal(B, K, V, dtype=dt).mul_(2.0 * T)
        likely = torch.randint(0, V, (B, K, 8), generator=gen, **dev)
        lift = T * (math.log(V) + 3.0 - 0.7 * torch.arange(8, **dev) + 0.3 * normal(B, K, 8, dtype=torch.float32))
        logits.scatter_(2, likely, lift.to(dt))
        # hypotheses of some length; some have ended; token 2 ends one
        scores = -20.0 - 2.0 * torch.rand(B, K, generator=gen, **dev)
        s.update(logits=logits, scores=scores, finished=cuda((rng.random((B, K)) < 0.125).astype(np.int32)), eos=2)
        return s
    Hkv, D, page, ctx = case["Hkv"], case["D"], case["page"], case["ctx"]
    blk = _block_bytes(case)
    if op in ("fork", "compact"):
        length = rng.integers(max(1, ctx // 2), ctx + 1, size=B).astype(np.int32)
        group = 8  # beams of one request share the first half of the first one's pages
        W = (ctx + case.get("grow", 0) + page - 1) // page + 1
        table = np.full((B, W), -1, np.int32)
        n_pages = int(B * W + case["spare"])
        ids = rng.permutation(n_pages)
        at = 0
        for b in range(B):
            n = -(-int(length[b]) // page)
            first = b - b % group
            shared = 0 if b == first else min(int(length[b]) // page, int(length[first]) // page) // 2
            table[b, :shared] = table[first, :shared]
            table[b, shared:n] = ids[at: at + n - shared]
            at += n - shared
        pages = torch.randint(0, 256, (case["planes"], n_pages, Hkv, blk), dtype=torch.uint8, generator=gen, **dev)
        s.update(pages=pages, table=cuda(table), length=cuda(length))
        if op == "fork":
            B2 = case["B2"]
            parent = (np.arange(B2) // group * group + rng.integers(0, group, size=B2)).clip(max=B - 1).astype(np.int32)
            parent[rng.random(B2) < 0.05] = -1  # requests that ended
            need = np.where(parent >= 0, length[parent] + rng.integers(1, case["grow"] + 1, size=B2), 0).astype(np.int32)
            s.update(parent=cuda(parent), need=cuda(need))
        return s
    N = case["N"]
    exps = cuda(np.stack([rng.integers(-3, 2, size=case.get("layers", 1)), rng.integers(-5, 1, size=case.get("layers", 1))],
                         axis=1).astype(np.int32))
    # committed lengths between half of ctx and ctx, the root among them
    base = rng.integers(max(1, ctx // 2), ctx + 1, size=B).astype(np.int32)
    W = (ctx + N + page - 1) // page
    n_pages = B * W + 3
    table = cuda(rng.permutation(n_pages)[: B * W].reshape(B, W).astype(np.int32))
    layers = case.get("layers", 1)
    pages = torch.zeros(layers, n_pages, Hkv, blk, dtype=torch.uint8, **dev)
    kc, ks, vc, vs = _parts(pages, page, D)
    for layer in range(layers):  # keys and values of the committed positions, a few hundred pages at a time
        for p0 in range(0, n_pages, 512):
            n = min(512, n_pages - p0)
            for c, sc, j in ((kc, ks, 0), (vc, vs, 1)):
                code, scale = _encode(normal(n, Hkv, page, D).float() * (1.0 if j == 0 else 0.5), exps[layer, j])
                c[layer, p0: p0 + n], sc[layer, p0: p0 + n] = code.unflatten(2, (-1, 16)), scale.unflatten(2, (-1, 16))
    chain = case.get("chain", not case.get("path", False))
    par, dep, anc = _trees(rng, B, N, 8, chain) if not chain else (None, None, None)
    s.update(pages=pages, table=table, base=cuda(base), exps=exps)
    if op == "attention":
        s.update(q=normal(B, N, Hkv * case["G"], D), nk=normal(B, N, Hkv, D), nv=0.5 * normal(B, N, Hkv, D),
                 scale=1.0 / math.sqrt(D), mask=None if chain else cuda(_pack(anc)))
        return s
    L = ctx + N
    s.update(nk=normal(layers, B, N, Hkv, D), nv=0.5 * normal(layers, B, N, Hkv, D), accepted=None, path=None,
             k=torch.zeros(layers, B, L, Hkv, D, dtype=torch.bfloat16, **dev),
             v=torch.zeros(layers, B, L, Hkv, D, dtype=torch.bfloat16, **dev))
    if case["path"]:
        path = np.full((B, 9), -1, np.int32)
        acc = np.zeros(B, np.int32)
        for b in range(B):
            node = int(rng.integers(0, N))
            acc[b] = dep[b, node]
            for d in range(acc[b], -1, -1):
                path[b, d] = node
                node = int(par[b, node])
        s.update(accepted=cuda(acc), path=cuda(path))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_attention(s):
    import speculative_decoding_verification_56_gb300 as sv
    q = s["q"]
    if "ws" not in s:  # kept by a decoding loop, with the outputs
        s["ws"] = sv.alloc_tree_attention_kv4_workspace(q, s["pages"][0])
        s["out"] = (torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device="cuda"))
    out, lse = s["out"]
    sv.spec_tree_attention_kv4(q, s["pages"][0], s["table"], s["nk"], s["nv"], s["mask"], s["base"], s["scale"], out, lse,
                               s["ws"], kv_exp=s["exps"][0])
    return dict(out=out, lse=lse)


def _own_store(s):
    import speculative_decoding_verification_56_gb300 as sv
    c = s["case"]
    if "ws" not in s:
        s["ws"] = sv.alloc_workspace(sv.SPEC_MODE_KV4, c["B"], c["N"], 1, sv.SPEC_DTYPE_BF16)
        s["len"] = torch.empty(c["B"], dtype=torch.int32, device="cuda")
    sv.spec_kv4_commit_path(s["pages"], s["table"], s["nk"], s["nv"], s["base"], s["accepted"], s["path"], s["len"], s["ws"],
                            kv_exp=s["exps"])
    sv.spec_kv4_read(s["pages"], s["table"], s["len"], s["k"], s["v"], s["ws"], kv_exp=s["exps"])
    return dict(new_len=s["len"], k=s["k"], v=s["v"])


def _own_fork(s):
    import speculative_decoding_verification_56_gb300 as sv
    if "ws" not in s:
        s["ws"] = sv.alloc_kv_pages_workspace(s["pages"], s["parent"].numel(), s["table"].shape[1])
        s["out"] = (torch.empty(s["parent"].numel(), s["table"].shape[1], dtype=torch.int32, device="cuda"),
                    torch.empty_like(s["parent"]), torch.empty(1, dtype=torch.int32, device="cuda"))
    table, length, used = s["out"]
    sv.spec_kv_pages_fork(s["pages"], s["table"], s["length"], s["parent"], s["need"], s["case"]["page"], table, length, used,
                          s["ws"])
    return dict(table=table, length=length, used=used, pages=s["pages"])


def _own_compact(s):
    import speculative_decoding_verification_56_gb300 as sv
    if "ws" not in s:
        s["ws"] = sv.alloc_kv_pages_workspace(s["pages"], *s["table"].shape)
        s["out"] = (torch.empty_like(s["table"]), torch.empty(1, dtype=torch.int32, device="cuda"))
    table, used = s["out"]
    sv.spec_kv_pages_compact(s["pages"], s["table"], table, used, s["ws"])
    return dict(table=table, used=used, pages=s["pages"])


def _own_beam(s):
    import speculative_decoding_verification_56_gb300 as sv
    c = s["case"]
    if "ws" not in s:
        B, K, V = s["logits"].shape
        i32 = dict(dtype=torch.int32, device="cuda")
        s["ws"] = sv.alloc_beam_select_workspace(s["logits"], c["M"])
        s["out"] = (torch.empty(B, c["M"], device="cuda"), torch.empty(B, c["M"], **i32), torch.empty(B, c["M"], **i32),
                    torch.empty(B, c["M"], **i32))
    scores, parents, tokens, finished = s["out"]
    sv.spec_beam_select(s["logits"], s["scores"], s["finished"], s["eos"], c["T"], scores, parents, tokens, finished, s["ws"])
    return dict(scores=scores, parents=parents, tokens=tokens, finished=finished)


def _gathered(s, layer):
    """Keys and values of every position that the table names, float32 [B, L, Hkv, D]."""
    c = s["case"]
    page, D = c["page"], c["D"]
    kc, ks, vc, vs = (x[layer] for x in _parts(s["pages"], page, D))
    at = s["table"].long()

    def take(codes, scales, e):
        y = _decode(codes[at], scales[at], e)  # [B, W, Hkv, page / 16, 16, D]
        return y.permute(0, 1, 3, 4, 2, 5).flatten(1, 3)

    return take(kc, ks, s["exps"][layer, 0]), take(vc, vs, s["exps"][layer, 1])


def _plain_attention(s):
    c = s["case"]
    B, N, Hkv, G, D = (c[k] for k in ("B", "N", "Hkv", "G", "D"))
    k, v = _gathered(s, 0)
    L = k.shape[1]
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) * s["scale"]
    node = torch.arange(N, device="cuda")
    if s["mask"] is None:
        tree = (node[None, :] <= node[:, None]).expand(B, N, N)
    else:
        tree = (s["mask"].long()[:, :, node // 32] >> (node % 32)) & 1 != 0
    z = q @ k.permute(0, 2, 3, 1)
    z.masked_fill_((torch.arange(L, device="cuda") >= s["base"][:, None] - 1)[:, None, None, :], -math.inf)
    zn = (q @ s["nk"].float().permute(0, 2, 3, 1)).view(B, Hkv, N, G, N)
    zn = zn.masked_fill(~tree[:, None, :, None, :], -math.inf).view(B, Hkv, N * G, N)
    m = torch.maximum(z.amax(3, keepdim=True), zn.amax(3, keepdim=True))
    e, en = (z - m).exp_(), (zn - m).exp_()
    total = e.sum(3, keepdim=True) + en.sum(3, keepdim=True)
    o = e @ v.permute(0, 2, 1, 3) + en @ s["nv"].float().permute(0, 2, 1, 3)
    out = (o / total).view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, D)
    lse = (m + total.log()).view(B, Hkv, N, G).permute(0, 2, 1, 3).reshape(B, N, Hkv * G)
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _plain_store(s):
    c = s["case"]
    B, N, page, D, layers = c["B"], c["N"], c["page"], c["D"], c["layers"]
    rows = torch.arange(B, device="cuda")[:, None]
    if s["path"] is None:
        node, last = torch.arange(N, device="cuda").expand(B, N), torch.full((B,), N - 1, device="cuda")
    else:
        node, last = s["path"].long(), s["accepted"].long()
    step = torch.minimum(torch.arange(node.shape[1], device="cuda").expand_as(node), last[:, None])  # (the last one again behind it)
    node = node.gather(1, step)
    at = s["base"].long()[:, None] - 1 + step
    pid, slot = s["table"].long().gather(1, at // page), at % page
    parts = _parts(s["pages"], page, D)
    new_len = s["base"] + last.int()
    L = s["k"].shape[2]
    seen = (torch.arange(L, device="cuda") < new_len[:, None])[:, :, None, None]
    for layer in range(layers):
        for j, x in ((0, s["nk"]), (1, s["nv"])):
            code, scale = _encode(x[layer][rows, node].float(), s["exps"][layer, j])
            parts[2 * j][layer].permute(0, 2, 3, 1, 4)[pid, slot // 16, slot % 16] = code
            parts[2 * j + 1][layer].permute(0, 2, 3, 1, 4)[pid, slot // 16, slot % 16] = scale
        for y, out in zip(_gathered(s, layer), (s["k"], s["v"])):
            out[layer] = torch.where(seen, y[:, :L].to(torch.bfloat16), out[layer])
    return dict(new_len=new_len, k=s["k"], v=s["v"])


def _plain_fork(s):
    c = s["case"]
    page, W, n_pages = c["page"], s["table"].shape[1], s["pages"].shape[1]
    B2 = s["parent"].numel()
    parent = s["parent"].long()
    length = torch.where(parent >= 0, s["length"].long()[parent.clamp(min=0)], 0)
    old = s["table"].long()[parent.clamp(min=0)]
    place, row = torch.arange(W, device="cuda"), torch.arange(B2, device="cuda")
    full, part = length // page, length % page > 0
    carried = place < full[:, None]
    open_ = torch.where(part, old.gather(1, full.clamp(max=W - 1)[:, None])[:, 0], n_pages)  # the unfinished page
    closed = torch.zeros(n_pages + 1, dtype=torch.bool, device="cuda")
    closed[torch.where(carried, old, n_pages)] = True
    lowest = torch.full((n_pages + 1,), B2, device="cuda").scatter_reduce_(0, open_, row, "amin")
    keep = part & ~closed[open_] & (lowest[open_] == row)
    closed[torch.where(keep, open_, n_pages)] = True
    kept = full + keep
    pages = torch.where(parent >= 0, (torch.maximum(s["need"].long(), length) + page - 1) // page, 0)
    fresh = pages - kept
    free = torch.sort(closed[:n_pages].byte(), stable=True).indices
    rank = (fresh.cumsum(0) - fresh)[:, None] + place - kept[:, None]
    table = torch.where(place < kept[:, None], old, free[rank.clamp(0, n_pages - 1)])
    table = torch.where(place < pages[:, None], table, -1)
    # rows without a copy copy a page that is in use onto itself
    copy = part & ~keep
    idle = closed[:n_pages].byte().argmax()
    src = torch.where(copy, open_, idle)
    dst = torch.where(copy, table.gather(1, full.clamp(max=W - 1)[:, None])[:, 0], idle)
    s["pages"][:, dst] = s["pages"][:, src]
    used = (closed[:n_pages].sum() + fresh.sum()).int().view(1)
    return dict(table=table.int(), length=length.int(), used=used, pages=s["pages"])


def _plain_compact(s):
    n_pages = s["pages"].shape[1]
    table = s["table"].long()
    held = torch.zeros(n_pages + 1, dtype=torch.bool, device="cuda")
    held[torch.where(table >= 0, table, n_pages)] = True
    held = held[:n_pages]
    used = held.sum()
    ids = torch.arange(n_pages, device="cuda")
    moves = held & (ids >= used)
    free = torch.sort(held.byte(), stable=True).indices  # the free places, in order
    to = torch.where(moves, free[(moves.cumsum(0) - 1).clamp(min=0)], ids)
    new = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    idle = torch.where(held & ~moves, ids, n_pages).amin().clamp(max=n_pages - 1)  # a page that stays
    src = torch.where(moves, ids, idle)
    dst = torch.where(moves, to, idle)
    for plane in s["pages"]:
        plane[dst] = plane[src]
    return dict(table=new.int(), used=used.int().view(1), pages=s["pages"])


def _plain_beam(s):
    """64 bits: candidates of different beams may lie close together."""
    c = s["case"]
    B, K, V = s["logits"].shape
    z = s["logits"].double() / c["T"]
    m = z.amax(2, keepdim=True)
    lse = m + (z - m).exp_().sum(2, keepdim=True).log_()
    total = z.sub_(lse).add_(s["scores"].double()[:, :, None])
    done = s["finished"] != 0
    total.masked_fill_(done[:, :, None], -math.inf)
    total[:, :, s["eos"]] = torch.where(done, s["scores"].double(), total[:, :, s["eos"]])
    total = total.view(B, K * V)
    scores, at = [], []
    for _ in range(c["M"]):
        best, i = total.max(1)
        scores.append(best)
        at.append(i)
        total.scatter_(1, i[:, None], -math.inf)
    scores, at = torch.stack(scores, 1), torch.stack(at, 1)
    some = scores > -math.inf
    beam, token = at // V, at % V
    ended = done.gather(1, beam) | (token == s["eos"])
    row = torch.arange(B, device="cuda")[:, None] * K + beam
    return dict(scores=scores.float(), parents=torch.where(some, row, -1).int(), tokens=torch.where(some, token, -1).int(),
                finished=(ended | ~some).int())


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, B = case["op"], case["B"]
    if op == "beam":
        size = 2 if case["dtype"] == "bf16" else 4
        rows = B * case["K"] * 0.875  # a finished beam's logits are not looked at
        return dict(bytes=rows * case["V"] * size + B * (8 * case["K"] + 16 * case["M"]), flops=rows * case["V"] * 4)
    D, Hkv, page = case["D"], case["Hkv"], case["page"]
    entry = Hkv * D * 9 // 8  # of one position, keys and values
    if op == "attention":
        N, Hq = case["N"], Hkv * case["G"]
        held = B * 0.75 * case["ctx"]
        W = 0 if case["chain"] else (N + 31) // 32
        moved = held * (entry + 4 / page) + B * N * (Hkv * D * 4 + Hq * D * 4 + Hq * 4 + 4 * W) + 4 * B
        return dict(bytes=moved, flops=4 * (N * held + B * N * min(N, 5)) * Hq * D)
    if op == "store":
        new = B * (5 if case["path"] else case["N"])
        held = B * 0.75 * case["ctx"] + new
        moved = case["layers"] * (new * (Hkv * D * 4 + entry) + held * (entry + Hkv * D * 4))
        return dict(bytes=moved, flops=case["layers"] * (new * 6 + held * 2) * Hkv * D)
    whole = case["planes"] * page * entry  # a page, all planes
    W = (case["ctx"] + case.get("grow", 0)) // page + 1
    if op == "fork":
        copies = 0.95 * case["B2"] * (1 - 1 / page) * 0.35  # takers that are not their parent's first
        return dict(bytes=2 * copies * whole + 4 * (B + case["B2"]) * W, flops=case["B2"] * W)
    held = B * 0.75 * case["ctx"] / page * 0.8
    moves = held * (1 - held / (case["spare"] + B * (W + 1)))  # pages that lie above the number held
    return dict(bytes=2 * moves * whole + 8 * B * W, flops=B * W)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers: nothing is rounded
    s = prepare(case, seed)
    return {"attention": _exact_attention, "store": _exact_store, "beam": _exact_beam}[case["op"]](case, s)


def _e4m3(b):
    """Value of an 8-bit scale: 4 exponent bits (bias 7), 3 of fraction."""
    e, f = (b >> 3) & 15, (b & 7).double()
    return torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)


def _exact_values(c, s, layer, b, n, j):
    """Keys (j = 0) or values of positions [0, n) of a sequence, float64 [n, Hkv, D]."""
    page, D = c["page"], c["D"]
    block = s["pages"][layer][s["table"][b, : -(-n // page)].long()].long()
    block = block.reshape(*block.shape[:2], page // 16, 2, 9 * D)[:, :, :, j]
    codes = block[..., : 8 * D].reshape(*block.shape[:2], page, D // 2)
    scales = block[..., 8 * D:].reshape(*block.shape[:2], page, D // 16)
    x = torch.empty(*codes.shape[:3], D, dtype=torch.float64, device="cuda")
    for k in (0, 1):
        y = (codes >> (4 * k)) & 15
        e, f = (y >> 1) & 3, (y & 1).double()
        mag = torch.where(e > 0, (2 + f) * torch.exp2(e.double() - 2), f / 2)
        x[..., k::2] = torch.where(y >= 8, -mag, mag)
    x = x * _e4m3(scales).repeat_interleave(16, -1) * 2.0 ** int(s["exps"][layer, j])
    return x.transpose(1, 2).reshape(-1, x.shape[1], D)[:n]


def _exact_attention(c, s):
    B, N, Hkv, G, D = (c[k] for k in ("B", "N", "Hkv", "G", "D"))
    out = torch.empty(B, N, Hkv * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, N, Hkv * G, dtype=torch.float64, device="cuda")
    bits = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        n = int(s["base"][b]) - 1
        sees = np.tril(np.ones((N, N), bool)) if bits is None else np.array(
            [[bits[b, v, w // 32] >> (w % 32) & 1 for w in range(N)] for v in range(N)], bool)
        hidden = torch.zeros(N, n + N, dtype=torch.bool, device="cuda")
        hidden[:, n:] = ~torch.from_numpy(sees).cuda()
        k = torch.cat([_exact_values(c, s, 0, b, n, 0), s["nk"][b].double()])
        v = torch.cat([_exact_values(c, s, 0, b, n, 1), s["nv"][b].double()])
        for h in range(Hkv * G):
            z = s["q"][b, :, h].double() @ k[:, h // G].T * s["scale"]
            z[hidden] = -math.inf
            lse[b, :, h] = torch.logsumexp(z, 1)
            out[b, :, h] = torch.softmax(z, 1) @ v[:, h // G]
    return dict(out=out, lse=lse)


def _nearest(x, grid):
    """Nearest of an ascending grid of magnitudes, ties to the even place."""
    x = x.clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, hi - 1)]


def _exact_rounded(x, e):
    """What x float64 [..., D] stands as in the pages."""
    steps = _e4m3(torch.arange(127, device="cuda"))
    codes = torch.tensor(CODES, dtype=torch.float64, device="cuda")
    y = x.unflatten(-1, (-1, 16)) * 2.0 ** -e
    # a / 6 against a grid: a against six times the grid, which is exact
    s = _nearest(y.abs().amax(-1, keepdim=True), 6 * steps) / 6
    s = steps[torch.searchsorted(steps, s - 1e-6 * s)]
    m = torch.where(s > 0, _nearest(y.abs() / s.clamp(min=2.0 ** -9), codes), 0)
    return (torch.where(y < 0, -m, m) * s).flatten(-2) * 2.0 ** e


def _exact_store(c, s):
    N = c["N"]
    k, v = s["k"].double(), s["v"].double()
    new_len = np.zeros(c["B"], np.int32)
    for b in range(c["B"]):
        start = int(s["base"][b]) - 1
        nodes = list(range(N)) if s["path"] is None else s["path"][b, : int(s["accepted"][b]) + 1].tolist()
        new_len[b] = start + len(nodes)
        for layer in range(c["layers"]):
            for j, x, out in ((0, s["nk"], k), (1, s["nv"], v)):
                out[layer, b, :start] = _exact_values(c, s, layer, b, start, j)
                out[layer, b, start: start + len(nodes)] = _exact_rounded(x[layer, b, nodes].double(), int(s["exps"][layer, j]))
    return dict(new_len=new_len, k=k, v=v)


def _exact_beam(c, s):
    B, K, V = s["logits"].shape
    M, eos = c["M"], s["eos"]
    out = dict(scores=np.full((B, M), -np.inf), parents=np.full((B, M), -1, np.int32), tokens=np.full((B, M), -1, np.int32),
               finished=np.ones((B, M), np.int32))
    for b in range(B):
        found = []
        for k in range(K):
            score = float(s["scores"][b, k])
            if int(s["finished"][b, k]):
                found.append((-score, k, eos, 1))
                continue
            p = torch.log_softmax(s["logits"][b, k].double() / c["T"], 0)
            value, token = torch.sort(p, descending=True, stable=True)
            for x, t in zip(value[:M].tolist(), token[:M].tolist()):
                found.append((-(score + x), k, t, int(t == eos)))
        for i, (x, k, t, f) in enumerate(sorted(found)[:M]):
            out["scores"][b, i], out["parents"][b, i], out["tokens"][b, i], out["finished"][b, i] = -x, b * K + k, t, f
    return out
