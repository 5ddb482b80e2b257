"""GPU parity of the tree's verification forward (head norms with rotation and
cache write, tree attention, tree sampling), through the C ABI, against the
float64 oracle.

Tolerances count roundings.  A rounding to bf16 is off by at most 2^-8 of the
value.  Attention rounds the softmax weights and the output to bf16, so an
output element differs by at most 2^-8 (|o| + A), A = sum_j w_j |v_j| (the same
attention over |v|), plus what float32 sums leave; a head element after norm
and rotation by 2^-8 |y| plus a few 2^-22 of the rotated pair.
"""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build, synth

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8     # largest relative error of a rounding to bf16
F32 = 2.0 ** -24     # and to float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()
    sv.load_library()
    oracle.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def parents_of(rng, B, N, max_depth=8, max_children=4):
    return np.stack([synth.make_tree_parents(rng, N, max_depth=max_depth,
                                             max_children=max_children)
                     for _ in range(B)]).astype(np.int32)


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------
# head norms, rotation, cache write
# ---------------------------------------------------------------------------

def check_qkv(B, N, Hq, Hkv, D, rot, interleaved, norm, chain=False, L=None, offset=0, seed=0,
              pad=0):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    L = L or N + 40
    qkv = randn(gen, B, N, Hq + 2 * Hkv, D) * 3
    qw = 1 + 0.2 * randn(gen, D) if norm else None
    kw = 1 + 0.2 * randn(gen, D) if norm else None
    inv = torch.from_numpy((10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32))
    base = rng.integers(1, L - N + 2, size=B).astype(np.int32)
    depth = None
    if not chain:
        depth = oracle.tree_mask(parents_of(rng, B, N))[1]
    kc = randn(gen, B, L + pad, Hkv, D)[:, :L]
    vc = randn(gen, B, L + pad, Hkv, D)[:, :L]
    k0, v0 = kc.clone(), vc.clone()
    q = sv.tree_qkv_rope(qkv, qw, kw, 1e-6, inv.cuda(), torch.from_numpy(base).cuda(),
                         None if chain else torch.from_numpy(depth).cuda(), kc, vc,
                         pos_offset=offset, interleaved=interleaved)
    torch.cuda.synchronize()
    qo, ko, vo = oracle.tree_qkv(bits(qkv), None if qw is None else bits(qw),
                                 None if kw is None else bits(kw), np.float32(1e-6), inv.numpy(),
                                 base, depth, Hkv, L, offset, interleaved)
    # a rotated element is made of two; the pair's size bounds its float32 error
    x = qkv.double().cpu().numpy()
    if norm:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True)) * 2
    pair = 2 * np.abs(x).max(axis=-1, keepdims=True)
    got = q.double().cpu().numpy()
    assert (np.abs(got - qo) <= BF16 * np.abs(qo) + 2.0 ** -20 * pair[:, :, :Hq]).all()
    kn, vn = kc.double().cpu().numpy(), vc.double().cpu().numpy()
    written = ~np.isnan(ko)
    for b in range(B):
        sl = slice(base[b] - 1, base[b] - 1 + N)
        assert (np.abs(kn[b, sl] - ko[b, sl]) <=
                BF16 * np.abs(ko[b, sl]) + 2.0 ** -20 * pair[b, :, Hq:Hq + Hkv]).all()
        assert (vn[b, sl] == vo[b, sl]).all()
    assert (kn[~written] == k0.double().cpu().numpy()[~written]).all()
    assert (vn[~written] == v0.double().cpu().numpy()[~written]).all()


@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot,interleaved,norm", [
    (1, 1, 1, 1, 64, 64, False, False),
    (2, 7, 8, 2, 128, 128, False, True),
    (3, 60, 32, 8, 128, 128, False, True),
    (5, 9, 15, 3, 64, 32, True, False),
    (2, 5, 6, 6, 128, 32, False, True),
    (2, 5, 7, 1, 128, 6, False, True),      # halves that are not whole vectors
    (2, 5, 7, 7, 64, 6, True, True),
    (2, 5, 4, 2, 64, 62, False, True),
    (4, 3, 5, 5, 64, 0, False, True),       # norm only
    (4, 3, 71, 1, 64, 64, False, False),    # one key head, an odd number of query heads
])
def test_qkv(B, N, Hq, Hkv, D, rot, interleaved, norm):
    check_qkv(B, N, Hq, Hkv, D, rot, interleaved, norm, seed=N + D + rot)


def test_qkv_chain_and_padded_cache():
    check_qkv(3, 5, 8, 2, 64, 64, False, True, chain=True, seed=3, pad=9)


def test_qkv_far_positions():
    # positions of ten million: the angle is still reduced exactly
    check_qkv(2, 4, 8, 2, 128, 128, False, False, offset=10_000_000, seed=5)


def test_qkv_tree_that_does_not_fit_is_left_alone():
    B, N, Hq, Hkv, D, L = 4, 6, 4, 2, 64, 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    qkv = randn(gen, B, N, Hq + 2 * Hkv, D)
    kc, vc = randn(gen, B, L, Hkv, D), randn(gen, B, L, Hkv, D)
    k0, v0 = kc.clone(), vc.clone()
    base = torch.tensor([0, L - N + 1, L - N + 2, -5], dtype=torch.int32, device="cuda")
    depth = torch.zeros(B, N, dtype=torch.int32, device="cuda")
    depth[1, 3] = -1
    ws = sv.alloc_workspace(sv.SPEC_MODE_TREE_QKV, B, N, 1, sv.SPEC_DTYPE_BF16)
    inv = torch.ones(D // 2, device="cuda")
    q = sv.tree_qkv_rope(qkv, None, None, 1e-6, inv, base, depth, kc, vc, workspace=ws)
    torch.cuda.synchronize()
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PATH | sv.SPEC_FLAG_BAD_PARENT
    for b in (0, 2, 3):
        assert (kc[b] == k0[b]).all() and (vc[b] == v0[b]).all() and (q[b] == 0).all()
    assert (vc[1, L - N:] == qkv[1, :, Hq + Hkv:]).all() and (kc[1, :L - N] == k0[1, :L - N]).all()
    assert torch.isfinite(q[1]).all()


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------

def check_attention(B, N, Hq, Hkv, D, base, P=0, chain=False, L=None, seed=0, pad=0, mask=None,
                    junk=True, spread=1.0, with_lse=True):
    """Runs one call and compares every output; returns (out, lse, flags).  With
    `junk`, everything that no node sees holds NaN or infinities."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    base = np.asarray(base, np.int32)
    L = L or int(base.max()) - 1 + N + 3
    q = randn(gen, B, N, Hq, D) * spread
    kc, vc = randn(gen, B, L + pad, Hkv, D), randn(gen, B, L + pad, Hkv, D)
    if mask is None and not chain:
        mask = oracle.tree_mask(parents_of(rng, B, N))[0]
    if junk:
        for b in range(B):
            end = base[b] - 1 + N
            kc[b, end:], vc[b, end:] = float("nan"), float("nan")
            vc[b, end:, :, ::2] = float("inf")
    pk = pv = None
    if P:
        pk, pv = randn(gen, P, Hkv, D), randn(gen, P, Hkv, D)
    ws = sv.alloc_tree_attention_workspace(q, kc, pk)
    scale = 1.0 / np.sqrt(D)
    maskd = None if mask is None else torch.from_numpy(mask.view(np.int32)).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    sv.spec_tree_attention(q, kc[:, :L], vc[:, :L], maskd, torch.from_numpy(base).cuda(), scale,
                           out, lse if with_lse else None, ws, prefix_k=pk, prefix_v=pv)
    torch.cuda.synchronize()
    flags = sv.spec_verify_read_flags(ws)
    kn, vn = bits(kc[:, :L]), bits(vc[:, :L])
    args = (bits(q), kn, vn, mask, base, scale)
    pre = (None, None) if pk is None else (bits(pk), bits(pv))
    o_ref, l_ref = oracle.tree_attention(*args, *pre)
    absv = (kn, vn & 0x7FFF)
    a_ref, _ = oracle.tree_attention(bits(q), *absv, mask, base, scale, pre[0],
                                     None if pk is None else pre[1] & 0x7FFF)
    # float32: the products' sums move a weight by D 2^-24 scale |q||k|, the
    # sums over the entries by their number times 2^-24
    reach = P + int(base.max()) + N
    kmax = float(kc[:, :L].float().nan_to_num(0, 0, 0).abs().amax()) if L else 0.0
    if P:
        kmax = max(kmax, float(pk.float().abs().amax()))
    qsum = float(q.float().abs().sum(-1).max())
    eps = F32 * (2 * D * scale * qsum * kmax + 2 * reach + 16)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = BF16 * (np.abs(o_ref) + a_ref) * (1 + 2.0 ** -6) + 2 * eps * a_ref
    assert (np.abs(got - o_ref) <= tol).all(), np.abs(got - o_ref).max()
    if with_lse:
        gl = lse.double().cpu().numpy()
        none = np.isneginf(l_ref)
        assert (np.isneginf(gl) == none).all()
        assert (np.abs(gl - l_ref)[~none] <= eps + 2 * F32 * np.abs(l_ref[~none])).all()
    return out, lse, flags


@pytest.mark.parametrize("B,N,Hq,Hkv,D,base,P,chain", [
    (1, 1, 1, 1, 64, [1], 0, True),                       # the root alone
    (1, 1, 4, 1, 128, [2], 0, True),
    (2, 5, 8, 8, 64, [301, 17], 0, True),
    (3, 1, 8, 2, 128, [128, 129, 130], 0, True),          # prefixes of 127, 128, 129 entries
    (2, 33, 8, 2, 128, [257, 1], 0, False),
    (3, 60, 8, 2, 128, [200, 1, 640], 0, False),          # rows of two tiles
    (2, 64, 12, 4, 64, [385, 100], 0, False),
    (2, 20, 15, 3, 128, [150, 260], 0, False),            # 5 heads share one
    (1, 9, 71, 1, 64, [333], 0, False),                   # 71 heads share one
    (1, 3, 128, 1, 64, [140], 0, False),
    (2, 200, 6, 2, 64, [70, 515], 0, False),              # more nodes than one item's rows
    (5, 4, 8, 2, 128, [1, 130, 7, 64, 1000], 257, False), # a shared prefix
    (3, 1, 4, 4, 64, [1, 1, 1], 1, True),                 # and nothing else
    (40, 7, 8, 2, 64, [20] * 40, 129, False),             # rows of many sequences in one tile
    (1, 2, 4, 1, 128, [20001], 0, True),                  # one long sequence
])
def test_attention(B, N, Hq, Hkv, D, base, P, chain):
    _, _, flags = check_attention(B, N, Hq, Hkv, D, base, P, chain, seed=B * N + D)
    assert flags == 0


def test_attention_cache_of_one_position():
    check_attention(1, 1, 8, 4, 128, [1], L=1, chain=True)
    check_attention(3, 2, 2, 2, 64, [1, 1, 1], L=2, chain=True)


def test_attention_large_logits():
    # weights from 1 down to nothing: running maxima grow far over many tiles
    check_attention(2, 6, 8, 2, 128, [900, 411], spread=24.0, seed=9)


def test_attention_padded_cache_without_lse():
    check_attention(3, 6, 8, 2, 64, [300, 20, 150], seed=4, pad=11, with_lse=False)


def test_attention_masks_that_leave_rows_empty():
    B, N = 2, 37
    mask = np.zeros((B, N, 2), np.uint32)
    mask[0, 5, 1] = 1 << 3          # node 5 sees node 35 only
    mask[0, 6] = 0xFFFFFFFF         # all nodes, and bits past the last node
    out, lse, flags = check_attention(B, N, 4, 2, 64, [1, 1], mask=mask, seed=2)
    assert flags == 0
    empty = torch.ones(B, N, dtype=torch.bool)
    empty[0, 5] = empty[0, 6] = False
    assert (out.cpu()[empty] == 0).all() and torch.isneginf(lse.cpu()[empty]).all()
    # with a prefix of its own, sequence 1 has something to see
    check_attention(B, N, 4, 2, 64, [1, 30], mask=mask, seed=2)


def test_attention_hidden_branches_may_hold_anything():
    """Entries of other branches hold NaN and infinities: each node's output is
    that of its own path alone."""
    B, N, Hq, Hkv, D = 1, 9, 4, 2, 64
    par = np.array([[-1, 0, 0, 1, 1, 2, 2, 3, 5]], np.int32)
    mask = oracle.tree_mask(par)[0]
    gen = torch.Generator(device="cuda").manual_seed(3)
    base, L = 150, 170
    q = randn(gen, B, N, Hq, D)
    kc, vc = randn(gen, B, L, Hkv, D), randn(gen, B, L, Hkv, D)
    maskd = torch.from_numpy(mask.view(np.int32)).cuda()
    based = torch.tensor([base], dtype=torch.int32, device="cuda")
    clean, clean_lse = sv.tree_attention(q, kc, vc, maskd, based)
    for n in range(N):
        k2, v2 = kc.clone(), vc.clone()
        for u in range(N):
            if not (mask[0, n, 0] >> u) & 1:
                k2[0, base - 1 + u] = float("nan") if u % 2 else float("inf")
                v2[0, base - 1 + u] = float("inf") if u % 2 else float("nan")
        out, lse = sv.tree_attention(q, k2, v2, maskd, based)
        torch.cuda.synchronize()
        assert (out[0, n] == clean[0, n]).all() and (lse[0, n] == clean_lse[0, n]).all()


def test_attention_entries_that_are_not_finite_stay_with_their_nodes():
    """An infinite value or key of a tree entry spoils the nodes that see it and
    no other, whatever tile or half they are in."""
    B, N, Hq, Hkv, D, base = 2, 150, 4, 2, 64, 101
    rng = np.random.default_rng(6)
    par = parents_of(rng, B, N)
    mask = oracle.tree_mask(par)[0]
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, kc = randn(gen, B, N, Hq, D), randn(gen, B, 300, Hkv, D)
    vc = randn(gen, B, 300, Hkv, D)
    maskd = torch.from_numpy(mask.view(np.int32)).cuda()
    based = torch.tensor([base, base + 77], dtype=torch.int32, device="cuda")
    clean, clean_lse = sv.tree_attention(q, kc, vc, maskd, based)
    for what, u in (("v", 40), ("v", 120), ("k", 130), ("v", 149)):
        k2, v2 = kc.clone(), vc.clone()
        (v2 if what == "v" else k2)[0, base - 1 + u, 1, 3] = float("inf")
        out, lse = sv.tree_attention(q, k2, v2, maskd, based)
        torch.cuda.synchronize()
        sees = torch.from_numpy((mask[0, :, u // 32] >> (u % 32)) & 1 != 0)
        assert 0 < sees.sum() < N
        assert (out[1] == clean[1]).all() and (lse[1] == clean_lse[1]).all()
        assert (out[0, :, :2] == clean[0, :, :2]).all()          # heads of the other key head
        assert (out[0, ~sees] == clean[0, ~sees]).all()
        # a score of -inf (an infinite key against a negative query element) is a
        # weight of 0; every other case spoils the head
        none = (q[0, :, 2:, 3] < 0) & (what == "k")
        assert (torch.isfinite(out[0, :, 2:]).all(dim=-1) == none)[sees].all()


def reference_attention(q, k, v, see, scale, pk=None, pv=None):
    """float64 on the GPU, sequence by sequence; `see` [B, N, L] truth values."""
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    out, lse = torch.zeros(B, N, Hq, D, dtype=torch.float64), torch.zeros(B, N, Hq, dtype=torch.float64)
    big = torch.zeros(B, N, Hq, D, dtype=torch.float64)
    for b in range(B):
        for h in range(Hq):
            kk, vv, ss = k[b, :, h // (Hq // Hkv)].double(), v[b, :, h // (Hq // Hkv)].double(), see[b]
            if pk is not None:
                kk = torch.cat([pk[:, h // (Hq // Hkv)].double(), kk])
                vv = torch.cat([pv[:, h // (Hq // Hkv)].double(), vv])
                ss = torch.cat([torch.ones(N, len(pk), dtype=torch.bool, device=ss.device), ss], 1)
            z = (q[b, :, h].double() @ kk.T * scale).masked_fill(~ss, float("-inf"))
            w = torch.softmax(z, 1)
            out[b, :, h], big[b, :, h], lse[b, :, h] = (w @ vv).cpu(), (w @ vv.abs()).cpu(), torch.logsumexp(z, 1).cpu()
    return out, big, lse


@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,P,chain", [
    (24, 1, 16, 4, 128, 4000, 0, True),      # decoding: runs of tiles over several sequences
    (9, 60, 32, 8, 128, 2500, 0, False),     # rows of two tiles, items cut anywhere
    (33, 12, 8, 8, 64, 1700, 1000, False),   # a shared prefix beside own ones
    (300, 2, 8, 1, 64, 90, 0, True),         # many short sequences
    (2, 500, 8, 2, 128, 3000, 0, True),      # long chains: several items per sequence
])
def test_attention_many_tiles(B, N, Hq, Hkv, D, ctx, P, chain):
    rng = np.random.default_rng(B)
    gen = torch.Generator(device="cuda").manual_seed(B)
    base = torch.from_numpy(rng.integers(1, ctx + 1, B).astype(np.int32)).cuda()
    L = ctx + N
    q, k, v = randn(gen, B, N, Hq, D), randn(gen, B, L, Hkv, D), randn(gen, B, L, Hkv, D)
    pk = randn(gen, P, Hkv, D) if P else None
    pv = randn(gen, P, Hkv, D) if P else None
    node = torch.arange(N, device="cuda")
    mask, tree = None, (node[None] <= node[:, None]).expand(B, N, N)
    if not chain:
        words, _, _ = oracle.tree_mask(parents_of(rng, B, N))
        mask = torch.from_numpy(words.view(np.int32)).cuda()
        tree = ((mask.long()[:, :, node // 32] >> (node % 32)) & 1) != 0
    see = torch.zeros(B, N, L, dtype=torch.bool, device="cuda")
    for b in range(B):
        p0 = int(base[b]) - 1
        see[b, :, :p0] = True
        see[b, :, p0:p0 + N] = tree[b]
    out, lse = sv.tree_attention(q, k, v, mask, base, prefix_k=pk, prefix_v=pv)
    torch.cuda.synchronize()
    want, big, wl = reference_attention(q, k, v, see, D ** -0.5, pk, pv)
    eps = F32 * (2 * D * D ** -0.5 * float(q.float().abs().sum(-1).max()) * 6 + 2 * (ctx + P + N))
    err = (out.double().cpu() - want).abs()
    assert (err <= BF16 * (want.abs() + big) * (1 + 2.0 ** -6) + 2 * eps * big).all(), err.max()
    assert ((lse.double().cpu() - wl).abs() <= eps + 2 * F32 * wl.abs()).all()


def test_attention_tree_that_does_not_fit():
    B, N, Hq, Hkv, D, L = 4, 6, 4, 2, 64, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = randn(gen, B, N, Hq, D)
    kc, vc = randn(gen, B, L, Hkv, D), randn(gen, B, L, Hkv, D)
    pk, pv = randn(gen, 40, Hkv, D), randn(gen, 40, Hkv, D)
    base = torch.tensor([0, L - N + 1, L - N + 2, 1 << 30], dtype=torch.int32, device="cuda")
    ws = sv.alloc_tree_attention_workspace(q, kc, pk)
    out, lse = sv.tree_attention(q, kc, vc, None, base, prefix_k=pk, prefix_v=pv, workspace=ws)
    torch.cuda.synchronize()
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PATH
    for b in (0, 2, 3):
        assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
    good, good_lse = sv.tree_attention(q[1:2].contiguous(), kc[1:2], vc[1:2], None, base[1:2],
                                       prefix_k=pk, prefix_v=pv)
    torch.cuda.synchronize()
    assert (out[1].float() - good[0].float()).abs().max() <= 2 * BF16 * good.float().abs().max()
    assert (lse[1] - good_lse[0]).abs().max() < 1e-4


def test_attention_is_repeatable_and_shares_a_workspace():
    """The same bits in every run, on a workspace that other shapes use in
    between and that starts out full of NaN bits."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, kc, vc = randn(gen, 6, 10, 8, 128), randn(gen, 6, 900, 2, 128), randn(gen, 6, 900, 2, 128)
    q2, kc2 = randn(gen, 3, 40, 8, 64), randn(gen, 3, 500, 4, 64)
    base = torch.tensor([800, 5, 640, 129, 1, 333], dtype=torch.int32, device="cuda")
    base2 = torch.tensor([300, 1, 450], dtype=torch.int32, device="cuda")
    n = max(sv.alloc_tree_attention_workspace(q, kc).numel(),
            sv.alloc_tree_attention_workspace(q2, kc2).numel())
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    first = [t.clone() for t in sv.tree_attention(q, kc, vc, None, base, workspace=ws)]
    for _ in range(3):
        sv.tree_attention(q2, kc2, kc2, None, base2, workspace=ws)
        again = sv.tree_attention(q, kc, vc, None, base, workspace=ws)
        torch.cuda.synchronize()
        assert (again[0] == first[0]).all() and (again[1] == first[1]).all()


# ---------------------------------------------------------------------------
# tree sampling
# ---------------------------------------------------------------------------

def tree_case(B, N, V, dtype, depth=6, T=1.0, seed=0, sigma=2.0):
    """Trees whose children hold likely tokens of their parent's row, so that
    walks go several nodes deep."""
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((B, N, V)) * sigma).astype(np.float32)
    par = parents_of(rng, B, N, max_depth=depth)
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        kids = {}
        for v in range(1, N):
            p = par[b, v]
            r = kids.get(p, 0)
            kids[p] = r + 1
            tok[b, v] = (p * 7919 + r * 31 + 5) % V
            z[b, p, tok[b, v]] = T * (np.log(V) + sigma ** 2 / 2 + 2.5 - 0.6 * r)
    tok[:, 0] = -1
    logits = sv.to_device_logits(z if dtype == "f32" else synth.f32_to_bf16_bits(z), dtype)
    host = bits(logits) if dtype == "bf16" else logits.cpu().numpy()
    u = rng.random((B, depth + 1)).astype(np.float32)
    u[u >= 1] = 0.5
    return logits, host, tok, par, u


def check_sample(logits, host, tok, par, u, T, depth, dtype):
    ws = sv.alloc_workspace(sv.SPEC_MODE_TREE_SAMPLE, *host.shape,
                            sv.SPEC_DTYPE_BF16 if dtype == "bf16" else sv.SPEC_DTYPE_F32)
    r = sv.verify_tree_sample(logits, torch.from_numpy(tok).cuda(), torch.from_numpy(par).cuda(),
                              torch.from_numpy(u).cuda(), T, depth, workspace=ws)
    torch.cuda.synchronize()
    o = oracle.verify_tree_sample(host, tok, par, u, np.float32(T), depth, dtype=dtype)
    # a draw closer to a border than the float64 sums' own error decides nothing
    clear = (o["margin"] > 1e-10) | (u == 0).any(axis=1)
    assert clear.all(), o["margin"]
    for key in ("accepted_len", "path_nodes", "out_tokens"):
        assert (r[key].cpu().numpy() == o[key]).all(), key
    got = r["out_probs"].double().cpu().numpy()
    # a weight and the total, each within 8e-6 of the total's float32 sum, and a rounding
    assert (np.abs(got - o["out_probs"]) <= (2 * 8e-6 + F32) * o["out_probs"]).all()
    return o, sv.spec_verify_read_flags(ws)


@pytest.mark.parametrize("B,N,V,dtype,T", [
    (1, 1, 1, "f32", 1.0), (2, 3, 2, "bf16", 1.0), (3, 8, 7, "f32", 0.5), (4, 20, 1000, "bf16", 1.0),
    (4, 20, 1001, "bf16", 1.0), (4, 20, 1003, "f32", 0.75), (3, 33, 4096, "f32", 1.5),
    (3, 12, 32003, "bf16", 1.0), (2, 12, 40000, "bf16", 1.0), (2, 10, 128256, "bf16", 0.75),
    (2, 5, 151937, "f32", 1.0), (1, 2, 400000, "bf16", 1.0), (1, 2, 1100000, "bf16", 1.0),
    (150, 6, 500, "f32", 1.0), (2, 1500, 30, "f32", 1.0),
])
def test_sample(B, N, V, dtype, T):
    c = tree_case(B, N, V, dtype, T=T, seed=B + N + V)
    o, flags = check_sample(*c, T, 6, dtype)
    assert flags == 0
    if B >= 3 and N >= 8:
        assert 0 < o["accepted_len"].sum()


def test_sample_largest_vocabulary():
    V = 1 << 26
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = randn(gen, 1, 1, V) * 3
    one = np.zeros((1, 1), np.int32)
    for u in (0.123, 0.987654):
        check_sample(logits, bits(logits), one, one - 1, np.array([[u]], np.float32), 1.0, 0, "bf16")


def test_sample_uniforms_at_the_ends():
    logits, host, tok, par, u = tree_case(3, 10, 3000, "bf16", seed=3)
    u[0], u[1], u[2] = 0.0, np.float32(1 - 2.0 ** -24), np.float32(2.0 ** -149)
    r = sv.verify_tree_sample(logits, torch.from_numpy(tok).cuda(), torch.from_numpy(par).cuda(),
                              torch.from_numpy(u).cuda(), 1.0, 6)
    torch.cuda.synchronize()
    assert (r["out_tokens"][0, 0] == 0) and (r["out_tokens"][2, 0] == 0)
    o = oracle.verify_tree_sample(host, tok, par, u, 1.0, 6)
    assert (r["out_tokens"].cpu().numpy() == o["out_tokens"]).all()


def test_sample_masked_vocabulary_and_empty_rows():
    logits, host, tok, par, u = tree_case(4, 10, 5000, "f32", seed=4)
    logits[0, :, 100:] = float("-inf")          # a grammar that allows 100 tokens
    logits[1, 0] = float("-inf")                # nothing at all
    logits[2, 0, :] = float("-inf")
    logits[2, 0, 4999] = -3.0                   # one token
    host = logits.cpu().numpy()
    o, flags = check_sample(logits, host, tok, par, u, 1.0, 6, "f32")
    assert flags == sv.SPEC_FLAG_EMPTY_ROW
    assert o["out_tokens"][1, 0] == -1 and o["out_tokens"][2, 0] == 4999
    assert (o["out_tokens"][0] < 100).all()


def test_sample_malformed_and_deep_trees():
    logits, host, tok, par, u = tree_case(2, 12, 300, "f32", depth=5, seed=5)
    par[0, 4], par[0, 5], tok[1, 3], par[1, 7] = 9, -3, 300, 7
    tok[0, 4] = tok[0, 5] = 5
    ws = sv.alloc_workspace(sv.SPEC_MODE_TREE_SAMPLE, 2, 12, 300, sv.SPEC_DTYPE_F32)
    args = (logits, torch.from_numpy(tok).cuda(), torch.from_numpy(par).cuda())
    r = sv.verify_tree_sample(*args, torch.from_numpy(u).cuda(), 1.0, 5, workspace=ws)
    torch.cuda.synchronize()
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PARENT | sv.SPEC_FLAG_TOKEN_RANGE
    o = oracle.verify_tree_sample(host, tok, par, u, 1.0, 5, dtype="f32")
    assert (r["path_nodes"].cpu().numpy() == o["path_nodes"]).all()
    # a chain of certain tokens, cut at the depth that the call allows
    z = torch.full((1, 6, 50), -1e4, device="cuda")
    z[:, :, 7] = 0.0
    chain = torch.tensor([[-1, 0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    sevens = torch.full((1, 6), 7, dtype=torch.int32, device="cuda")
    for depth, want, flag in ((3, 3, sv.SPEC_FLAG_DEPTH), (0, 0, sv.SPEC_FLAG_DEPTH), (5, 5, 0), (9, 5, 0)):
        r = sv.verify_tree_sample(z, sevens, chain, torch.full((1, depth + 1), 0.5, device="cuda"),
                                  1.0, depth, workspace=ws)
        torch.cuda.synchronize()
        assert r["accepted_len"].item() == want
        assert r["out_tokens"][0].tolist() == [7] * (want + 1) + [-1] * (depth - want)
        assert sv.spec_verify_read_flags(ws) == flag


def test_sample_twin_children_take_the_first():
    z = torch.full((1, 5, 9), -50.0, device="cuda")
    z[0, 0, 4] = z[0, 1, 2] = z[0, 2, 3] = 10.0
    par = torch.tensor([[-1, 0, 0, 2, 1]], dtype=torch.int32, device="cuda")
    tok = torch.tensor([[0, 4, 4, 3, 2]], dtype=torch.int32, device="cuda")
    r = sv.verify_tree_sample(z, tok, par, torch.full((1, 4), 0.3, device="cuda"), 1.0, 3)
    assert r["path_nodes"].tolist() == [[0, 1, 4, -1]]


@pytest.mark.parametrize("V,dtype", [(64, "f32"), (1024, "bf16"), (65536, "bf16")])
def test_sample_draws_on_and_next_to_the_borders(V, dtype):
    """Equal logits: the borders are the multiples of 1 / V, and a uniform on one
    of them, or the floats beside it, falls where exact arithmetic says."""
    rng = np.random.default_rng(V)
    j = np.concatenate([[0, 1, V - 1], rng.integers(0, V, 60)])
    u = (j / V).astype(np.float32)
    assert (u.astype(np.float64) * V == j).all()      # V is a power of two: exact
    u = np.concatenate([u, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0))])
    n = len(u)
    logits = torch.full((n, 1, V), -3.25, device="cuda",
                        dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    one = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    r = sv.verify_tree_sample(logits, one, one - 1, torch.from_numpy(u[:, None]).cuda(), 0.75, 0)
    torch.cuda.synchronize()
    want = np.floor(u.astype(np.float64) * V).astype(np.int32)
    assert (r["out_tokens"].cpu().numpy()[:, 0] == want).all()


def test_sample_spread_out_logits():
    """Ranges of the logits far apart from one part of the row to the next, where
    references of the float32 sums lie hundreds of powers of two apart."""
    rng = np.random.default_rng(12)
    B, V = 12, 70000
    z = rng.standard_normal((B, 1, V)).astype(np.float32)
    at = np.arange(V)
    z[0:3] += 300.0 * np.sin(at / 9000.0)          # smooth, peaks of many near-equal weights
    z[3:6] += -4000.0 * (at // 4096 != 7)          # one part holds all the mass
    z[6] = -1e6 + 0.01 * z[6]
    z[7] = 2e6 + np.round(z[7])
    z[8, 0, ::2] = -np.inf
    z[9, 0, 5:] = -np.inf
    z[10, 0, :4096] += 30.0                        # the first elements are the largest
    z[11, 0, 300:] += 150.0                        # the first elements are far too small
    u = rng.random((B, 1)).astype(np.float32)
    u[u >= 1] = 0.5
    one = np.zeros((B, 1), np.int32)
    logits = torch.from_numpy(z).cuda()
    o, flags = check_sample(logits, z, one, one - 1, u, 1.0, 0, "f32")
    assert flags == 0


def test_sample_law_of_the_first_token():
    """Over many uniforms the first token follows softmax(z / T) (chi-square)."""
    V, n, T = 40, 20000, 0.75
    rng = np.random.default_rng(8)
    z = (rng.standard_normal(V) * 1.2).astype(np.float32)
    u = ((np.arange(n) + rng.random(n)) / n).astype(np.float32)   # stratified
    logits = torch.from_numpy(z).cuda().expand(n, 1, V).contiguous()
    one = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    r = sv.verify_tree_sample(logits, one, one - 1, torch.from_numpy(u[:, None]).cuda().contiguous(), T, 0)
    p = np.exp(z.astype(np.float64) / T)
    p /= p.sum()
    counts = np.bincount(r["out_tokens"].cpu().numpy()[:, 0], minlength=V)
    # a stratified sample misses each border by at most one of n
    assert np.abs(counts - n * p).max() <= 2


# ---------------------------------------------------------------------------
# the three together, and their use of streams and graphs
# ---------------------------------------------------------------------------

class TinyModel:
    """One attention layer over cached keys and values, with an LM head."""

    def __init__(self, V=600, Hq=4, Hkv=2, D=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.V = Hq, Hkv, D, V
        self.emb = randn(g, V, 128, dtype=torch.float32)
        self.wqkv = randn(g, 128, (Hq + 2 * Hkv) * D, dtype=torch.float32) / 11
        self.wo = randn(g, Hq * D, V, dtype=torch.float32) / 4
        self.qw, self.kw = 1 + 0.1 * randn(g, D), 1 + 0.1 * randn(g, D)
        self.inv = (10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)).float()

    def forward(self, tokens, base, depth, mask, kc, vc):
        B, N = tokens.shape
        qkv = (self.emb[tokens.long()] @ self.wqkv).bfloat16().view(B, N, -1, self.D)
        q = sv.tree_qkv_rope(qkv, self.qw, self.kw, 1e-6, self.inv, base, depth, kc, vc)
        out, _ = sv.tree_attention(q, kc, vc, mask, base)
        return (out.float().flatten(2) @ self.wo).contiguous()


def test_tree_steps_emit_what_one_by_one_decoding_emits():
    """Tree steps (mask, forward, sampling, KV commit) with any drafts emit the
    tokens that decoding one by one emits with the same uniforms."""
    m = TinyModel()
    B, N, L, steps, depth = 3, 14, 160, 12, 4
    rng = np.random.default_rng(1)
    dev = "cuda"
    first = torch.from_numpy(rng.integers(0, m.V, (B, 1)).astype(np.int32)).to(dev)
    uni = torch.from_numpy(rng.random((B, 200)).astype(np.float32)).to(dev)

    def caches():
        return (torch.zeros(2, B, L, m.Hkv, m.D, dtype=torch.bfloat16, device=dev)).unbind(0)

    # one by one
    kc, vc = caches()
    tok, base, plain = first, torch.ones(B, dtype=torch.int32, device=dev), []
    top2 = []
    for i in range(60):
        z = m.forward(tok, base, None, None, kc, vc)
        r = sv.verify_tree_sample(z, tok, tok * 0 - 1, uni[:, i:i + 1].contiguous(), 1.0, 0)
        plain.append(r["out_tokens"].clone())
        top2.append(z[:, 0].topk(3).indices)
        tok, base = r["out_tokens"].contiguous(), base + 1
    plain = torch.cat(plain, 1).cpu().numpy()
    # by trees whose children are sometimes what will be drawn
    cache = torch.zeros(2, B, L, m.Hkv, m.D, dtype=torch.bfloat16, device=dev)
    base, got, accepted = np.ones(B, np.int32), [[] for _ in range(B)], 0
    root = first.cpu().numpy()[:, 0]
    for _ in range(steps):
        par = parents_of(rng, B, N, max_depth=depth, max_children=3)
        mask_d, depth_d = sv.tree_attention_mask(torch.from_numpy(par).to(dev))
        toks = rng.integers(0, m.V, (B, N)).astype(np.int32)
        dep = depth_d.cpu().numpy()
        for b in range(B):
            for v in range(1, N):
                at = len(got[b]) + dep[b, v] - 1
                if rng.random() < 0.6 and at < plain.shape[1]:
                    toks[b, v] = plain[b, at]
        toks[:, 0] = root
        toks_d, base_d = torch.from_numpy(toks).to(dev), torch.from_numpy(base).to(dev)
        z = m.forward(toks_d, base_d, depth_d, mask_d, cache[0], cache[1])
        u = torch.stack([uni[b, len(got[b]): len(got[b]) + depth + 1] for b in range(B)]).contiguous()
        r = sv.verify_tree_sample(z, toks_d, torch.from_numpy(par).to(dev), u, 1.0, depth)
        new_len = torch.empty(B, dtype=torch.int32, device=dev)
        ws = sv.alloc_workspace(sv.SPEC_MODE_KV_COMMIT, B, N, 1, sv.SPEC_DTYPE_BF16)
        sv.spec_kv_commit_path(cache, base_d, r["accepted_len"], r["path_nodes"], N, new_len, ws)
        torch.cuda.synchronize()
        assert sv.spec_verify_read_flags(ws) == 0
        n, out = r["accepted_len"].cpu().numpy(), r["out_tokens"].cpu().numpy()
        accepted += int(n.sum())
        for b in range(B):
            got[b] += out[b, : n[b] + 1].tolist()
            root[b] = out[b, n[b]]
        base = new_len.cpu().numpy() + 1
    assert accepted > 10
    # logits of the two orders of work differ by roundings, which a draw next to
    # a border may show: after such a draw the texts go apart
    same = [int(np.argmin(np.append(np.array(g[:60]) == plain[b][: len(g)], False)))
            for b, g in enumerate(got)]
    assert sum(same) >= 0.9 * sum(min(60, len(g)) for g in got), same


def test_forward_on_a_side_stream_and_in_a_graph():
    m = TinyModel(seed=2)
    B, N, L = 2, 9, 700
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = randn(gen, 2, B, L, m.Hkv, m.D)
    par = torch.from_numpy(parents_of(rng, B, N)).cuda()
    mask, depth = sv.tree_attention_mask(par)
    qkv = randn(gen, B, N, m.Hq + 2 * m.Hkv, m.D)
    base = torch.tensor([400, 77], dtype=torch.int32, device="cuda")
    z = randn(gen, B, N, 1000, dtype=torch.float32) * 3
    tok = torch.from_numpy(rng.integers(0, 1000, (B, N)).astype(np.int32)).cuda()
    u = torch.rand(B, 5, generator=gen, device="cuda")
    q = torch.empty(B, N, m.Hq, m.D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, N, m.Hq, device="cuda")
    res = [torch.empty(B, dtype=torch.int32, device="cuda")] + \
          [torch.empty(B, 5, dtype=torch.int32, device="cuda") for _ in range(2)] + \
          [torch.empty(B, 5, device="cuda")]
    wa = sv.alloc_tree_attention_workspace(q, cache[0])
    wq = sv.alloc_workspace(sv.SPEC_MODE_TREE_QKV, B, N, 1, sv.SPEC_DTYPE_BF16)

    def step(stream=None):
        sv.spec_tree_qkv_rope(qkv, m.qw, m.kw, 1e-6, m.inv, base, depth, q, cache[0], cache[1], wq,
                              stream=stream)
        sv.spec_tree_attention(q, cache[0], cache[1], mask, base, 0.125, out, lse, wa, stream=stream)
        sv.spec_verify_tree_sample(z, tok, par, u, 1.0, 4, *res, wq, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (q, out, lse, *res)]
    side = torch.cuda.Stream()
    for t in (q, out, lse, *res):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all((a == b).all() for a, b in zip((q, out, lse, *res), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q, out, lse, *res):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all((a == b).all() for a, b in zip((q, out, lse, *res), want))
    # a replay reads the lengths of its own time
    base.copy_(torch.tensor([20, 650], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    torch.cuda.synchronize()
    assert (got == out).all() and not (got == want[1]).all()


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with a workspace of its own."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    cases = []
    for B, N, ctx, D in ((20, 30, 1500, 128), (7, 61, 900, 64)):
        q, kc, vc = randn(gen, B, N, 8, D), randn(gen, B, ctx + N, 2, D), randn(gen, B, ctx + N, 2, D)
        base = torch.randint(1, ctx, (B,), generator=gen, device="cuda", dtype=torch.int32)
        z = randn(gen, B, N, 5000)
        tok = torch.randint(0, 5000, (B, N), generator=gen, device="cuda", dtype=torch.int32)
        par = torch.arange(-1, N - 1, device="cuda", dtype=torch.int32).expand(B, N).contiguous()
        u = torch.rand(B, N, generator=gen, device="cuda")
        cases.append((q, kc, vc, base, z, tok, par, u))

    def run(c, stream=None):
        q, kc, vc, base, z, tok, par, u = c
        out, lse = sv.tree_attention(q, kc, vc, None, base, stream=stream)
        r = sv.verify_tree_sample(z, tok, par, u, 1.0, u.shape[1] - 1, stream=stream)
        return [out, lse, *r.values()]
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [run(c, s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_empty_batches_are_no_ops():
    kc = torch.zeros(0, 9, 2, 64, dtype=torch.bfloat16, device="cuda")
    base = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = sv.tree_qkv_rope(torch.zeros(0, 3, 8, 64, dtype=torch.bfloat16, device="cuda"), None, None, 1e-6, None,
                         base, None, kc, kc)
    assert q.shape == (0, 3, 4, 64)
    out, lse = sv.tree_attention(q, kc, kc, None, base)
    assert out.shape == q.shape and lse.shape == (0, 3, 4)
    i = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    r = sv.verify_tree_sample(torch.zeros(0, 3, 50, device="cuda"), i, i, torch.zeros(0, 3, device="cuda"), 1.0, 2)
    assert r["out_tokens"].shape == (0, 3)


def test_wrappers_refuse_what_does_not_fit():
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, kc = randn(gen, 2, 3, 4, 64), randn(gen, 2, 50, 2, 64)
    base = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sv.tree_attention(q, kc, kc[:, :40], None, base)
    with pytest.raises(ValueError):
        sv.tree_attention(q, kc, kc, None, base[:1])
    with pytest.raises(ValueError):
        sv.tree_attention(q, kc.transpose(1, 2).contiguous().transpose(1, 2), kc, None, base)
    with pytest.raises(TypeError):
        sv.tree_attention(q, kc.half(), kc.half(), None, base)
    with pytest.raises(ValueError):
        sv.tree_attention(q, kc, kc, None, base, prefix_k=kc[0])
    with pytest.raises(ValueError):
        sv.tree_attention(q, kc, kc, torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda"), base)
    with pytest.raises(sv.SpecVerifyError):
        sv.tree_attention(q, kc, kc, None, base, scale=0.0, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    z = randn(gen, 2, 3, 100)
    i = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sv.verify_tree_sample(z, i, i, torch.zeros(2, 3, device="cuda"), 1.0, 3)
    with pytest.raises(TypeError):
        sv.verify_tree_sample(z, i.long(), i, torch.zeros(2, 4, device="cuda"), 1.0, 3)
    with pytest.raises(ValueError):
        sv.verify_tree_sample(z, i, i.cpu(), torch.zeros(2, 4, device="cuda"), 1.0, 3)


def test_qkv_frequencies_of_many_turns():
    # more than 2^23 turns a position: the float below the product's first one
    # holds whole turns too.  At position 1 the angle is off by 2^-47 of it
    # (8e7 turns: 6e-7 of a turn, 4e-6), far below the roundings counted here
    N, D = 2, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    qkv = randn(gen, 1, N, 3, D)
    inv = torch.linspace(6e7, 5e8, D // 2)
    kc, vc = randn(gen, 1, 9, 1, D), randn(gen, 1, 9, 1, D)
    base = np.array([1], np.int32)
    q = sv.tree_qkv_rope(qkv, None, None, 1e-6, inv.cuda(), torch.from_numpy(base).cuda(), None, kc,
                         vc)
    torch.cuda.synchronize()
    qo, ko, _ = oracle.tree_qkv(bits(qkv), None, None, np.float32(1e-6), inv.numpy(), base, None, 1, 9)
    pair = 2 * float(qkv.float().abs().max())
    eps = (4e-6 + 2.0 ** -20) * pair
    assert (np.abs(q.double().cpu().numpy() - qo) <= BF16 * np.abs(qo) + eps).all()
    kn = kc.double().cpu().numpy()[:, :N]
    assert (np.abs(kn - ko[:, :N]) <= BF16 * np.abs(ko[:, :N]) + eps).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N,ctx", [(1, 5), (1, 700), (40, 300)])
def test_attention_scores_far_from_zero(N, ctx, sign):
    # every score is +-2^23 (64 products of 2^17): equal weights, so the output
    # is the mean of V, and the log-sum the score plus ln of their number
    D, Hkv, Hq = 64, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(ctx)
    q = torch.full((1, N, Hq, D), 2.0 ** 8, dtype=torch.bfloat16, device="cuda")
    kc = torch.full((1, ctx + N, Hkv, D), sign * 2.0 ** 9, dtype=torch.bfloat16, device="cuda")
    vc = randn(gen, 1, ctx + N, Hkv, D)
    base = torch.tensor([ctx + 1], dtype=torch.int32, device="cuda")
    out, lse = sv.tree_attention(q, kc, vc, None, base, scale=1.0)
    torch.cuda.synchronize()
    v = vc.double().cpu().numpy()[0]
    for n in range(N):
        seen = v[: ctx + 1 + n]
        mean = seen.mean(axis=0).repeat(Hq // Hkv, axis=0)
        mag = np.abs(seen).mean(axis=0).repeat(Hq // Hkv, axis=0)
        got = out[0, n].double().cpu().numpy()
        # a weight rounds to bf16 (all of them alike, 2^-8 of it), the output
        # once more; float32 sums of ctx + N terms
        tol = BF16 * (np.abs(mean) + mag) * (1 + 2.0 ** -6) + 2 * (ctx + N) * F32 * mag
        assert (np.abs(got - mean) <= tol).all()
        # the reference, its sum with log2 and the product with ln 2 round
        want = sign * 2.0 ** 23 + np.log(len(seen))
        assert (np.abs(lse[0, n].double().cpu().numpy() - want) <= 4 * F32 * 2.0 ** 23).all()


@pytest.mark.parametrize("raw", [False, True])
def test_conveniences_allocate_on_the_stream_of_the_call(raw):
    """A workspace that goes out of use when its call returns is not handed to
    another stream while the call is still to run."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    B, N, ctx = 3, 20, 1500
    q, kc, vc = randn(gen, B, N, 8, 64), randn(gen, B, ctx + N, 2, 64), randn(gen, B, ctx + N, 2, 64)
    base = torch.tensor([ctx, 3, 900], dtype=torch.int32, device="cuda")
    want, want_lse = sv.tree_attention(q, kc, vc, None, base)
    nbytes = sv.spec_tree_attention_workspace_bytes(B, N, 8, 2, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    out, lse = sv.tree_attention(q, kc, vc, None, base, stream=side.cuda_stream if raw else side)
    held = [torch.full((nbytes,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and len(held) == 3


@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,P", [
    (900, 2, 2, 1, 64, 60, 0),       # more sequences than one scan of the lengths takes
    (900, 1, 4, 2, 64, 150, 130),
    (1, 4096, 1, 1, 64, 100, 0),     # the largest tree
])
def test_attention_many_sequences_and_nodes(B, N, Hq, Hkv, D, ctx, P):
    base = np.random.default_rng(B + N).integers(1, ctx + 1, B)
    _, _, flags = check_attention(B, N, Hq, Hkv, D, base, P, chain=N < 3, seed=B, junk=False)
    assert flags == 0


def test_cache_offsets_past_32_bits():
    # two sequences 2^31 + 2^20 elements apart give what a compact cache gives
    B, N, Hq, Hkv, D, L = 2, 9, 8, 2, 64, 700
    step = (1 << 31) + (1 << 20)
    gen = torch.Generator(device="cuda").manual_seed(21)
    small = [randn(gen, B, L, Hkv, D) for _ in range(2)]
    far = []
    for t in small:
        flat = torch.empty(step + L * Hkv * D, dtype=torch.bfloat16, device="cuda")
        far.append(flat.as_strided((B, L, Hkv, D), (step, Hkv * D, D, 1)))
        far[-1].copy_(t)
    qkv = randn(gen, B, N, Hq + 2 * Hkv, D)
    inv = torch.linspace(1.0, 1e-4, D // 2, device="cuda")
    base = torch.tensor([33, 651], dtype=torch.int32, device="cuda")
    res = []
    for k, v in (small, far):
        q = sv.tree_qkv_rope(qkv, None, None, 1e-6, inv, base, None, k, v)
        res.append((q, *sv.tree_attention(q, k, v, None, base)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.equal(small[0], far[0]) and torch.equal(small[1], far[1])


def test_sample_rows_past_32_bits():
    # row 599 of V = 2^22 starts 2.5e9 elements in
    N, V = 600, 1 << 22
    z = torch.zeros(1, N, V, dtype=torch.bfloat16, device="cuda")
    z[0, 0, 12345] = z[0, N - 1, 777] = 40.0   # e^40 against 4e6: probability 1 to 2e-11
    tok = torch.arange(N, dtype=torch.int32, device="cuda")[None].contiguous()
    tok[0, N - 1] = 12345
    par = torch.zeros(1, N, dtype=torch.int32, device="cuda")
    u = torch.full((1, 2), 0.5, device="cuda")
    r = sv.verify_tree_sample(z, tok, par, u, 1.0, 1)
    torch.cuda.synchronize()
    assert r["accepted_len"].tolist() == [1] and r["path_nodes"].tolist() == [[0, N - 1]]
    assert r["out_tokens"].tolist() == [[12345, 777]]
    assert (r["out_probs"] - 1).abs().max() < 2e-5
