"""Edges of the tree's verification forward on the GPU: workspaces of exactly the
size asked for, values that are not finite, draws among very unlikely tokens,
waits that run out, and calls that the documentation allows at its limits."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build
from test_gpu_tree_forward import check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()
    sv.load_library()
    oracle.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


# ---------------------------------------------------------------------------
# the attention's workspace
# ---------------------------------------------------------------------------

def lengths(B, longest, seed, first=None):
    base = np.random.default_rng(seed).integers(1, longest + 1, B)
    if first:
        base[0] = first
    return base.tolist()


@pytest.mark.parametrize("B,N,Hq,Hkv,D,base,P", [
    (3, 9, 8, 2, 128, [900, 3, 400], 0),                     # few items: a slot by item
    (40, 7, 16, 8, 64, lengths(40, 900, 1), 0),              # 320 items: slots by CTA
    (170, 1, 2, 1, 64, lengths(170, 60, 2, first=30000), 0), # one of them over many CTAs
    (30, 40, 48, 8, 128, lengths(30, 300, 3), 0),            # rows of two tiles, by CTA
    (9, 5, 8, 2, 128, lengths(9, 500, 4), 300),              # own slots smaller than the prefix's
    (3, 1, 4, 4, 64, [1, 70, 200], 1000),
    (70, 3, 6, 2, 64, lengths(70, 200, 5), 129),
])
def test_attention_keeps_to_its_workspace(monkeypatch, B, N, Hq, Hkv, D, base, P):
    guard = 1 << 20
    held = []

    def exact(q, k_cache, prefix_k=None):
        n = sv.spec_tree_attention_workspace_bytes(*q.shape[:3], k_cache.shape[2], q.shape[3],
                                                   0 if prefix_k is None else prefix_k.shape[0])
        held.append((torch.full((n + guard,), 0xFF, dtype=torch.uint8, device="cuda"), n))
        held[-1][0][:4] = 0
        return held[-1][0][:n]

    monkeypatch.setattr(sv, "alloc_tree_attention_workspace", exact)
    _, _, flags = check_attention(B, N, Hq, Hkv, D, base, P, chain=N == 1, seed=B + N)
    buf, n = held[0]
    assert flags == 0 and len(held) == 1 and (buf[n:] == 0xFF).all()


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("N,D,P,base", [
    (9, 64, 0, [40, 3]),        # one tile: written by its only CTA
    (9, 128, 0, [700, 300]),    # halves by alternate tiles, items cut
    (70, 64, 0, [333, 900]),    # rows of two tiles
    (9, 64, 200, [150, 20]),    # joined with a shared prefix
    (70, 128, 130, [100, 1]),
])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_attention_values_that_are_not_finite(N, D, P, base, value):
    """One element of V: of a tree entry it makes the whole output NaN for the
    nodes that see it; of a committed entry or the prefix, its own column for all
    nodes.  The log-sums, which V has no part in, keep their bits."""
    rng = np.random.default_rng(N + D)
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    B, Hq, Hkv, L, col, head = 2, 4, 2, 1000, 5, 1

    def randn(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.bfloat16, device="cuda")

    q, kc, vc = randn(B, N, Hq, D), randn(B, L, Hkv, D), randn(B, L, Hkv, D)
    pk, pv = (randn(P, Hkv, D), randn(P, Hkv, D)) if P else (None, None)
    par = np.stack([np.concatenate([[-1], [rng.integers(0, v) for v in range(1, N)]]) for _ in range(B)])
    mask = oracle.tree_mask(par.astype(np.int32))[0]
    maskd = torch.from_numpy(mask.view(np.int32)).cuda()
    based = torch.tensor(base, dtype=torch.int32, device="cuda")
    clean, lse0 = sv.tree_attention(q, kc, vc, maskd, based, prefix_k=pk, prefix_v=pv)
    heads = slice(head * Hq // Hkv, (head + 1) * Hq // Hkv)
    for b in range(B):
        at = [base[b] - 1 + u for u in (0, N // 2, N - 1)] + [t for t in (0, base[b] - 2) if 0 <= t < base[b] - 1]
        for t in at:
            v2 = vc.clone()
            v2[b, t, head, col] = value
            out, lse = sv.tree_attention(q, kc, v2, maskd, based, prefix_k=pk, prefix_v=pv)
            want = clean.clone()
            u = t - (base[b] - 1)
            if u >= 0:
                sees = torch.from_numpy(mask[b, :, u // 32] >> (u % 32) & 1 != 0).cuda()
                assert sees.any()
                want[b, sees, heads] = float("nan")
            else:
                want[b, :, heads, col] = float("nan")
            spoilt = torch.isnan(want)
            assert torch.equal(lse, lse0)
            assert torch.equal(out[~spoilt], clean[~spoilt])
            assert not torch.isfinite(out[spoilt]).any()
            if u >= 0:
                assert torch.isnan(out[spoilt]).all()
    if P:
        p2 = pv.clone()
        p2[P - 1, head, col] = value
        out, lse = sv.tree_attention(q, kc, vc, maskd, based, prefix_k=pk, prefix_v=p2)
        assert torch.equal(lse, lse0) and not torch.isfinite(out[:, :, heads, col]).any()
        out[:, :, heads, col] = clean[:, :, heads, col]
        assert torch.equal(out, clean)


# ---------------------------------------------------------------------------
# tree sampling: draws among very unlikely tokens
# ---------------------------------------------------------------------------

def draw_first(logits, u, T=1.0):
    """The tokens that uniforms u draw from the one row `logits`."""
    rows = logits.expand(len(u), -1)[:, None].contiguous()
    one = torch.zeros(len(u), 1, dtype=torch.int32, device="cuda")
    r = sv.verify_tree_sample(rows, one, one - 1, torch.tensor(u, dtype=torch.float32, device="cuda")[:, None], T, 0)
    torch.cuda.synchronize()
    return r["out_tokens"].cpu().numpy()[:, 0].astype(np.float64), r["out_probs"].double().cpu().numpy()[:, 0]


@pytest.mark.parametrize("V,z,dtype", [
    (1 << 26, -24.625, torch.bfloat16),   # 1.4 times 2^-36 of the largest each, 1.4e-3 of it together
    (1 << 26, -27.5, torch.bfloat16),
    ((1 << 24) + 3, -26.25, torch.float32),
    (1 << 22, -27.5, torch.float32),      # 0.6 of 2^-39
])
@pytest.mark.parametrize("first", [True, False])
def test_sample_a_flat_tail_of_a_large_vocabulary(V, z, dtype, first):
    """One likely token and V - 1 alike: the borders are an arithmetic series, and
    a draw falls within V 2^-51 + 2^-28 of the total of where it should."""
    row = torch.full((1, V), z, dtype=dtype, device="cuda")
    row[0, 0 if first else V - 1] = 0.0
    w = float(np.exp(z))                    # (bf16 holds these z exactly)
    R = 1.0 + (V - 1) * w
    part = np.array([0.1, 0.37, 0.5, 0.93])
    u = ((1.0 + part * (R - 1)) / R if first else part * (R - 1) / R).astype(np.float32)
    x, p = draw_first(row, u)
    t = u.astype(np.float64) * R
    lo = np.where(x == 0, 0.0, 1.0 + (x - 1) * w) if first else x * w
    hi = 1.0 + x * w if first else np.where(x == V - 1, R, (x + 1) * w)
    off = (V * 2.0 ** -51 + 2.0 ** -28) * R
    assert (lo - off <= t).all() and (t < hi + off).all(), (lo - t, hi - t)
    likely = x == (0 if first else V - 1)
    want = np.where(likely, 1.0, w) / R
    assert (np.abs(p - want) <= 2e-5 * want).all()


@pytest.mark.parametrize("V", [1 << 20, 1 << 26])
def test_sample_borders_of_a_large_vocabulary(V):
    """Equal logits: a uniform on a border, or the float beside it, falls where
    exact arithmetic says (every sum is a multiple of one weight)."""
    rng = np.random.default_rng(V)
    j = np.array([1, V // 2, V - 64, *(rng.integers(0, 1 << 20, 4) * (V >> 20))])
    u = (j / V).astype(np.float32)
    assert (u.astype(np.float64) * V == j).all()
    for v in (u, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0))):
        x, _ = draw_first(torch.full((1, V), -3.25, dtype=torch.bfloat16, device="cuda"), v, T=0.75)
        assert (x == np.floor(v.astype(np.float64) * V)).all()


# ---------------------------------------------------------------------------
# the attention's waits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,P", [
    (20, 1, 8, 2, 128, 3000, 0),      # halves by alternate tiles
    (9, 60, 16, 4, 128, 2000, 0),     # rows of two tiles
    (16, 9, 8, 2, 64, 500, 1500),     # and a shared prefix
])
def test_attention_waits_that_run_out(B, N, Hq, Hkv, D, ctx, P):
    """A wait that takes longer than its limit ends the call with the flag set (1 ns:
    at the first wait that is not over at its first look; longer limits let the
    roles get further), and the next call is right."""
    gen = torch.Generator(device="cuda").manual_seed(B)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.bfloat16, device="cuda")

    q, kc, vc = randn(B, N, Hq, D), randn(B, ctx + N, Hkv, D), randn(B, ctx + N, Hkv, D)
    pk, pv = (randn(P, Hkv, D), randn(P, Hkv, D)) if P else (None, None)
    base = torch.randint(1, ctx, (B,), generator=gen, device="cuda", dtype=torch.int32)
    ws = sv.alloc_tree_attention_workspace(q, kc, pk)

    def call():
        out, lse = sv.tree_attention(q, kc, vc, None, base, prefix_k=pk, prefix_v=pv, workspace=ws)
        torch.cuda.synchronize()
        return out, lse, sv.spec_verify_read_flags(ws)

    want = call()
    assert want[2] == 0
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for limit in (1, 300, 1000, 3000, 10000, 10 ** 9):
        flush.fill_(1)                       # the copies come from memory, not from L2
        sv.spec_verify_set_wait_limit_ns(limit)
        try:
            out, lse, flags = call()
        finally:
            sv.spec_verify_set_wait_limit_ns(0)
        assert flags == (sv.SPEC_FLAG_TIMEOUT if limit == 1 else flags & sv.SPEC_FLAG_TIMEOUT)
        if limit == 10 ** 9:
            assert flags == 0
        if flags == 0:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        again = call()
        assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_attention_runs_of_long_items_are_not_given_up():
    """Each CTA has seven items of half a million entries, several ms each, one
    after the other: no role may take the time of a whole item for a wait that
    has run out (limit 1 ms)."""
    N, Hq, D, ctx = 2200, 128, 64, 512 * 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(1, N, Hq, D, generator=gen, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.randn(1, ctx + N, 1, D, generator=gen, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    base = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    ws = sv.alloc_tree_attention_workspace(q, kc)
    want = sv.tree_attention(q, kc, vc, None, base, workspace=ws)
    assert sv.spec_verify_read_flags(ws) == 0
    sv.spec_verify_set_wait_limit_ns(1_000_000)
    try:
        out, lse = sv.tree_attention(q, kc, vc, None, base, workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.spec_verify_set_wait_limit_ns(0)
    assert sv.spec_verify_read_flags(ws) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------
# calls that take what the call before them writes
# ---------------------------------------------------------------------------

def test_calls_chained_without_a_pause():
    """Mask, heads, attention, sampling and KV commit, each on the outputs of the
    one before, step after step with other trees and lengths and nothing in
    between: what the same calls give with a pause after each."""
    B, N, Hq, Hkv, D, L, V, depth, steps = 5, 24, 8, 2, 64, 400, 900, 6, 40
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, dtype=dtype, device="cuda")

    def ints(*shape):
        return torch.empty(*shape, dtype=torch.int32, device="cuda")

    par = torch.from_numpy(np.stack([[[-1] + [rng.integers(0, v) for v in range(1, N)] for _ in range(B)]
                                     for _ in range(steps)]).astype(np.int32)).cuda()
    tok = torch.from_numpy(rng.integers(0, 3, (steps, B, N)).astype(np.int32)).cuda()
    base = torch.from_numpy(rng.integers(1, L - N, (steps, B)).astype(np.int32)).cuda()
    qkv = randn(steps, B, N, Hq + 2 * Hkv, D)
    z = randn(steps, B, N, V, dtype=torch.float32)
    z[..., :3] += 8.0                      # the three tokens that nodes hold
    u = torch.rand(steps, B, depth + 1, generator=gen, device="cuda")
    inv = torch.linspace(1.0, 1e-3, D // 2, device="cuda")
    cache0 = randn(2, B, L, Hkv, D)

    def run(pause):
        cache, got = cache0.clone(), []
        ws = torch.zeros(max(sv.spec_tree_attention_workspace_bytes(B, N, Hq, Hkv, D), 256),
                         dtype=torch.uint8, device="cuda")
        mask, dep, q = ints(B, N, 1), ints(B, N), torch.empty(B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
        n, path, out_tok, new_len = ints(B), ints(B, depth + 1), ints(B, depth + 1), ints(B)
        prob = torch.empty(B, depth + 1, device="cuda")
        outs = torch.empty(steps, B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
        lens = ints(steps, B)
        for s in range(steps):
            calls = (lambda: sv.spec_tree_attention_mask(par[s], mask, dep, ws),
                     lambda: sv.spec_tree_qkv_rope(qkv[s], None, None, 1e-6, inv, base[s], dep, q, cache[0],
                                                   cache[1], ws),
                     lambda: sv.spec_tree_attention(q, cache[0], cache[1], mask, base[s], 0.125, outs[s], None, ws),
                     lambda: sv.spec_verify_tree_sample(z[s], tok[s], par[s], u[s], 1.0, depth, n, path, out_tok,
                                                        prob, ws),
                     lambda: sv.spec_kv_commit_path(cache, base[s], n, path, N, lens[s], ws))
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, lens, cache, sv.spec_verify_read_flags(ws)

    want = run(True)
    assert want[3] & ~sv.SPEC_FLAG_DEPTH == 0 and (want[1] > base).any()
    for _ in range(3):
        got = run(False)
        assert got[3] == want[3]
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))


# ---------------------------------------------------------------------------
# angles of far positions
# ---------------------------------------------------------------------------

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qkv_angles_are_as_exact_as_the_header_says(interleaved):
    """Pairs (1, 0) turn into (cos, sin) of position * frequency; an angle of A
    turns may be off by A 2^-47 + 2^-24 of a turn, and the outputs are rounded."""
    D, Hkv = 64, 1
    freq = np.exp(np.random.default_rng(5).uniform(np.log(1e-5), np.log(3000.0), D // 2)).astype(np.float32)
    freq[:4] = 1.0, 0.5, 100.0, 1e-4
    offset = 2 ** 31 - 1
    depth = torch.tensor([[0, 1, 2, 3, 77, 1000, 123456, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    N = depth.shape[1]
    qkv = torch.zeros(1, N, 1 + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    qkv[..., 0::2 if interleaved else 1][..., : D // 2] = 1.0
    kc = torch.zeros(1, N + 1, Hkv, D, dtype=torch.bfloat16, device="cuda")
    base = torch.tensor([2], dtype=torch.int32, device="cuda")
    q = sv.tree_qkv_rope(qkv, None, None, 1e-6, torch.from_numpy(freq).cuda(), base, depth, kc, kc.clone(),
                         pos_offset=offset, interleaved=interleaved).double().cpu().numpy()[0, :, 0]
    cos, sin = (q[:, 0::2], q[:, 1::2]) if interleaved else (q[:, : D // 2], q[:, D // 2:])
    for n in range(N):
        pos = offset + 1 + int(depth[0, n])
        for i, f in enumerate(freq):
            turns = pos * Fraction(float(f)) / (2 * PI)
            angle = 2 * np.pi * float(turns - round(turns))
            off = 2 * np.pi * (float(turns) * 2.0 ** -47 + 2.0 ** -24)
            # a rounding to bf16, and the float32 sine and cosine's own 2 ulp
            tol = 2.0 ** -8 + 2.0 ** -22
            for got, want in ((cos[n, i], np.cos(angle)), (sin[n, i], np.sin(angle))):
                assert abs(got - want) <= off + tol * (abs(want) + off), (n, i, got, want, off)
