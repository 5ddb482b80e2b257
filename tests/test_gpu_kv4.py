"""The 4-bit cache in pages on the GPU against 64-bit references: commit, read and
the tree's attention, alone and together with the calls around them."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()
    sv.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(rng, *shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * scale).bfloat16().cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def flags_of(ws):
    return sv.spec_verify_read_flags(ws, clear=True)


def random_pages(rng, n_pages, Hkv, page, D):
    """Any codes; scales whose keys and values are of the order of 1."""
    blk = rng.integers(0, 256, (n_pages, Hkv, page // 16, 2, 9 * D), dtype=np.uint8)
    blk[..., 8 * D:] = rng.integers(30, 50, blk[..., 8 * D:].shape, dtype=np.uint8)  # 2^-4.. of a code
    return blk.reshape(n_pages, Hkv, 9 * page * D // 8)


def tree_mask(rng, B, N, p_up=0.7):
    """Ancestor relations of random trees, and their words."""
    anc = np.zeros((B, N, N), bool)
    for b in range(B):
        for v in range(N):
            if v:
                par = v - 1 if rng.random() < p_up else int(rng.integers(0, v))
                anc[b, v] = anc[b, par]
            anc[b, v, v] = True
    return anc, pack_mask(anc)


def pack_mask(anc):
    B, N, _ = anc.shape
    W = (N + 31) // 32
    full = np.zeros((B, N, W * 32), np.uint8)
    full[:, :, :N] = anc
    return np.packbits(full, axis=2, bitorder="little").view(np.uint32).view(np.int32).reshape(B, N, W).copy()


class Case:
    """Inputs of the attention, and its 64-bit outputs."""

    def __init__(self, B, N, Hq, Hkv, D, page, base, chain, seed=0, exps=None, W=None, spare=3):
        rng = self.rng = np.random.default_rng(seed + 1000 * B + N)
        self.B, self.N, self.Hq, self.Hkv, self.D, self.page = B, N, Hq, Hkv, D, page
        W = W or max(1, max(-(-(b - 1) // page) for b in base))
        n_pages = B * W + spare
        self.table = rng.permutation(n_pages)[: B * W].reshape(B, W).astype(np.int32)
        self.pages = random_pages(rng, n_pages, Hkv, page, D)
        self.q, self.nk, self.nv = bf16(rng, B, N, Hq, D), bf16(rng, B, N, Hkv, D), bf16(rng, B, N, Hkv, D)
        self.base = np.array(base, np.int32)
        self.anc, words = (np.tril(np.ones((B, N, N), bool)), None) if chain else tree_mask(rng, B, N)
        self.words = words
        self.exps = exps
        self.scale = D ** -0.5

    def run(self, stream=None, workspace=None):
        ws = workspace
        if ws is None:
            ws = sv.alloc_tree_attention_kv4_workspace(self.q, cuda(self.pages))
        self.ws = ws
        return sv.tree_attention_kv4(
            self.q, cuda(self.pages), cuda(self.table), self.nk, self.nv,
            None if self.words is None else cuda(self.words), cuda(self.base), self.scale,
            None if self.exps is None else cuda(np.array(self.exps, np.int32)), ws, stream)

    def check(self, out, lse):
        """Errors: a score's sum of D products in float32, cut off at each
        addition, D 2^-23 of sum |q k|; the exponential and float32 sums of a
        row's weights, at most 600 of them in turn, 4e-5 in all; weights 2^-11
        (fp16), and as much twice more where a renewed reference scales stored
        ones by a factor in fp16; half a step of bf16, 2^-8.  fp16 has no steps
        below 2^-24, so that rounding is off by up to 2^-25 even of the smallest
        weights, which are held 2^7 times as large as against a reference of
        weight 1: an entry adds up to 2^-32 |v| over a total of at least 1."""
        out, lse = host(out), host(lse)
        assert not np.isnan(out).any() and not np.isnan(lse).any()
        for b in range(self.B):
            n = int(self.base[b]) - 1
            k, v = ref.unpack(self.pages, self.table[b], n, self.page, self.D, self.exps or (0, 0))
            k = np.concatenate([k, host(self.nk[b])])
            v = np.concatenate([v, host(self.nv[b])])
            sees = np.concatenate([np.ones((self.N, n), bool), self.anc[b]], 1)
            o, l, mass, amp = ref.attention(host(self.q[b]), k, v, sees, self.scale)
            ds = self.D * 2.0 ** -23 * amp + 4e-5
            none = np.isinf(l)
            assert (lse[b][none] == -np.inf).all() and (out[b][none] == 0).all()
            assert (np.abs(lse[b][~none] - l[~none]) <= ds[~none] + 2.0 ** -22 * np.abs(l[~none])).all()
            small = 2.0 ** -32 * np.repeat(np.abs(np.nan_to_num(v)).sum(0), self.Hq // self.Hkv, axis=0)
            tol = 2.0 ** -8 * np.abs(o) + (3 * 2.0 ** -11 + 2 * ds[..., None]) * mass + small
            worst = np.max(np.abs(out[b] - o) - tol)
            assert worst <= 1e-30, worst


SHAPES = [
    # few rows
    (3, 1, 4, 4, 64, 16, [1, 2, 17], True),
    (5, 1, 32, 8, 128, 64, [5000, 1, 129, 33, 257], True),
    (1, 5, 8, 8, 64, 16, [300], True),
    (2, 4, 8, 2, 64, 32, [300, 40], False),          # 16 rows
    (2, 3, 40, 5, 128, 128, [700, 1], False),        # 24 rows
    (1, 2, 10, 2, 128, 16, [4097], True),            # 10 rows
    (70, 1, 8, 2, 64, 32, list(range(1, 211, 3)), True),
    (300, 1, 2, 1, 64, 16, [1 + (7 * i) % 90 for i in range(300)], True),
    (1, 20, 1, 1, 128, 64, [513], True),             # one head
    # tiles of the tensor cores
    (2, 60, 32, 8, 128, 64, [3000, 100], False),
    (3, 33, 40, 8, 128, 128, [900, 1, 128], False),
    (2, 1, 128, 1, 64, 16, [40, 300], True),         # 128 heads of one
    (1, 300, 8, 8, 128, 32, [1], True),              # nodes alone, three tiles of them
    (1, 1500, 4, 2, 64, 64, [200], True),            # a chunk of a prompt
    (2, 26, 3, 3, 64, 16, [129, 128], False),        # 26 rows, the tree at a tile's edge
    (40, 13, 8, 2, 128, 16, [1 + 31 * i for i in range(40)], False),
    (2, 129, 2, 2, 128, 128, [130, 2], False),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,base,chain", SHAPES)
def test_attention(B, N, Hq, Hkv, D, page, base, chain):
    c = Case(B, N, Hq, Hkv, D, page, base, chain)
    out, lse = c.run()
    assert flags_of(c.ws) == 0
    c.check(out, lse)


@pytest.mark.parametrize("N,D", [(1, 64), (1, 128), (40, 64), (40, 128)])
@pytest.mark.parametrize("exps", [(3, -2), (-20, 30), (-64, 64), (64, -64)])
def test_attention_exponents(N, D, exps):
    """Keys and values far from 1: the cache's exponents scale the nodes too."""
    c = Case(2, N, 8, 2, D, 32, [150, 40], True, exps=exps)
    c.nk = (c.nk.float() * 2.0 ** exps[0]).bfloat16()
    c.nv = (c.nv.float() * 2.0 ** exps[1]).bfloat16()
    c.scale = D ** -0.5 * 2.0 ** -exps[0]
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("N,D", [(1, 64), (3, 128), (40, 128), (90, 64)])
def test_attention_large_and_growing_scores(N, D):
    """References are renewed, also in the middle of a tile, and far scores vanish."""
    c = Case(2, N, 4, 1, D, 64, [1000, 777], True, exps=(0, 0))
    c.scale = 2.0
    c.pages = c.pages.copy()
    blocks = c.pages.reshape(c.pages.shape[0], 1, 4, 2, 9 * D)
    for b in range(2):
        for i, pid in enumerate(c.table[b]):
            for g in range(4):  # scales grow along the sequence
                blocks[pid, 0, g, 0, 8 * D:] = 20 + (i * 4 + g) % 40
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("N", [1, 6, 50])
def test_attention_nodes_that_see_nothing(N):
    c = Case(2, N, 8, 2, 64, 16, [1, 40], False)
    c.anc = np.random.default_rng(N).random((2, N, N)) < 0.3
    c.anc[:, 0] = False
    c.words = pack_mask(c.anc)
    c.words[:, :, -1] |= np.int32(-(1 << (N % 32)) if N % 32 else 0)  # bits past N are not looked at
    out, lse = c.run()
    c.check(out, lse)
    assert (lse[0, 0] == -np.inf).all() and (out[0, 0] == 0).all()


@pytest.mark.parametrize("N,D,page", [(1, 128, 16), (2, 64, 64), (40, 128, 16), (40, 64, 128)])
def test_attention_positions_without_a_page(N, D, page):
    c = Case(2, N, 8, 2, D, page, [700, 300], True)
    c.table[0, 1], c.table[0, 3], c.table[1, 0] = -1, len(c.pages), 1 << 30
    out, lse = c.run()
    assert flags_of(c.ws) == sv.SPEC_FLAG_BAD_PAGE
    c.check(out, lse)


@pytest.mark.parametrize("N", [1, 40])
@pytest.mark.parametrize("bad", [0, -5, 200])
def test_attention_lengths_outside_the_table(N, bad):
    """Such a sequence gives 0 and -inf; the others are as they would be."""
    c = Case(3, N, 8, 2, 64, 16, [50, 60, 70], True, W=6)
    c.base[1] = bad
    out, lse = c.run()
    assert flags_of(c.ws) == sv.SPEC_FLAG_BAD_PATH
    assert (out[1] == 0).all() and (lse[1] == -np.inf).all()
    keep = [0, 2]
    c.B, c.base, c.table, c.anc = 2, c.base[keep], c.table[keep], c.anc[keep]
    c.q, c.nk, c.nv = c.q[keep], c.nk[keep], c.nv[keep]
    c.check(out[keep], lse[keep])


@pytest.mark.parametrize("N,D", [(6, 64), (6, 128), (60, 64), (150, 128)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("which", ["nk", "nv"])
def test_attention_nodes_that_are_not_finite(N, D, value, which):
    """They make NaN of the rows that see them, and of no other."""
    c = Case(2, N, 6, 3, D, 16, [90, 1], False)
    at = N // 2
    good_out, good_lse = c.run()
    setattr(c, which, getattr(c, which).clone())
    getattr(c, which)[0, at, 1, D - 3] = value
    out, lse = c.run()
    sees = c.anc[0, :, at]
    heads = [2, 3]
    for h in range(6):
        hit = sees if h in heads else np.zeros(N, bool)
        assert torch.isnan(out[0, hit, h]).all() and torch.isnan(lse[0, hit, h]).all()
        assert torch.equal(out[0, ~hit, h], good_out[0, ~hit, h])
        assert torch.equal(lse[0, ~hit, h], good_lse[0, ~hit, h])
    assert torch.equal(out[1], good_out[1]) and torch.equal(lse[1], good_lse[1])


@pytest.mark.parametrize("N", [2, 40])
def test_attention_query_that_is_not_finite(N):
    c = Case(1, N, 4, 2, 128, 16, [90], True)
    good, _ = c.run()
    c.q = c.q.clone()
    c.q[0, 1, 2, 5] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(lse[0, 1, 2])
    rest = torch.ones(N, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.equal(out[0][rest.cuda()], good[0][rest.cuda()])


@pytest.mark.parametrize("N", [1, 40])
def test_attention_tiny_huge_and_zero_queries(N):
    c = Case(1, N, 8, 2, 64, 16, [200], True)
    c.q = c.q.clone()
    c.q[0, 0, 0] *= 1e-30
    c.q[0, 0, 1] *= 2.0 ** 14
    c.q[0, 0, 2] = 0
    c.q[0, 0, 3, 7] *= 1e4
    c.q[0, 0, 4] = 1e-40
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("N", [1, 40])
def test_attention_stale_bytes_are_not_used(N):
    """Behind a sequence's last position its page may hold anything, as scales of
    NaN (0x7F); so may pages that the table does not name."""
    c = Case(2, N, 8, 2, 128, 64, [100, 65], True)
    want = c.run()
    used = set()
    for b in range(2):
        for t in range(int(c.base[b]) - 1):
            used.add((int(c.table[b, t // 64]), t % 64))
    groups = c.pages.reshape(len(c.pages), 2, 4, 2, 9 * 128)
    for pid in range(len(c.pages)):
        for slot in range(64):
            if (pid, slot) not in used:
                g, s = slot // 16, slot % 16
                groups[pid, :, g, :, s * 64: s * 64 + 64] = 0xFF
                groups[pid, :, g, :, 8 * 128 + s * 8: 8 * 128 + s * 8 + 8] = 0x7F
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_attention_pages_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes, and pages at its end."""
    Hkv, page, D, n_pages = 8, 128, 128, 30000
    pages = torch.zeros(n_pages, Hkv, 9 * page * D // 8, dtype=torch.uint8, device="cuda")
    assert pages.nbytes > 1 << 32
    for N in (1, 40):
        c = Case(1, N, 8, Hkv, D, page, [600], True)
        ids = n_pages - 1 - 2 * np.arange(c.table.shape[1])
        pages[cuda(ids).long()] = cuda(c.pages[c.table[0]])
        ws = sv.alloc_tree_attention_kv4_workspace(c.q, pages)
        out, lse = sv.tree_attention_kv4(c.q, pages, cuda(ids[None].astype(np.int32)), c.nk, c.nv, None,
                                         cuda(c.base), c.scale, None, ws)
        c.check(out, lse)


@pytest.mark.parametrize("B,N,Hq", [(40, 1, 8), (3, 2, 8), (9, 40, 8), (200, 30, 2)])
def test_attention_keeps_to_its_workspace(B, N, Hq):
    base = [1 + (97 * i) % 700 for i in range(B)]
    c = Case(B, N, Hq, 2, 64, 32, base, True)
    n = sv.spec_tree_attention_kv4_workspace_bytes(B, N, Hq, 2, 64)
    buf = torch.full((n + (1 << 20),), 0xFF, dtype=torch.uint8, device="cuda")
    buf[:4] = 0
    out, lse = c.run(workspace=buf[:n])
    assert (buf[n:] == 0xFF).all() and flags_of(buf[:n]) == 0
    c.check(out, lse)


@pytest.mark.parametrize("N", [1, 40])
def test_attention_on_other_streams_and_captured(N):
    """Two calls at once on two streams, and a captured one with new inputs: the
    same bits as one after the other."""
    cases = [Case(4, N, 8, 2, 128, 64, [900, 40, 1, 333], True, seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [c.run(stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = cases
    q, pages, table, nk, nv, base = (t.clone() for t in (a.q, cuda(a.pages), cuda(a.table), a.nk, a.nv, cuda(a.base)))
    ws = sv.alloc_tree_attention_kv4_workspace(q, pages)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_tree_attention_kv4(q, pages, table, nk, nv, None, base, a.scale, out, lse, ws)
    for c, w in ((a, want[0]), (b, want[1])):
        for t, x in zip((q, pages, table, nk, nv, base), (c.q, cuda(c.pages), cuda(c.table), c.nk, c.nv, cuda(c.base))):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("N,base", [(1, [3000] * 4), (1, [100000] * 3), (40, [3000] * 4)])
def test_attention_waits_that_run_out(N, base):
    """With a limit of one look the call ends, with the flag where it had to wait
    (the roles for one another; copies may have landed before they are looked at)
    and right where not; the next one is right."""
    c = Case(len(base), N, 8, 2, 128, 64, base, True)
    sv.spec_verify_set_wait_limit_ns(1)
    try:
        first = c.run()
        torch.cuda.synchronize()
        flags = flags_of(c.ws)
        assert flags == sv.SPEC_FLAG_TIMEOUT or (flags == 0 and N == 1)
    finally:
        sv.spec_verify_set_wait_limit_ns(0)
    out, lse = c.run()
    assert flags_of(c.ws) == 0
    if flags == 0:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    if max(base) <= 3000:
        c.check(out, lse)


# ---------------------------------------------------------------------------
# commit and read
# ---------------------------------------------------------------------------

def values(rng, *shape):
    """bf16 of many magnitudes, some at borders of two codes, some 0."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-12, 12, shape[:-1] + (1,))
    grid = rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]), shape)
    tie = rng.random(shape[:-1] + (1,)) < 0.3  # blocks with 6 and borders: scale 1 or a power of two
    x = np.where(tie, grid * np.sign(x), x)
    x[rng.random(shape) < 0.05] = 0
    x[(rng.random(shape[:-1]) < 0.03)] = 0
    return torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()


@pytest.mark.parametrize("layers,B,N,Hkv,D,page", [
    (1, 1, 1, 1, 64, 16), (2, 3, 7, 3, 64, 16), (3, 2, 60, 8, 128, 64), (1, 5, 33, 5, 128, 128), (2, 1, 700, 2, 64, 32),
])
@pytest.mark.parametrize("kind", ["path", "chain", "all"])
def test_commit_and_read(layers, B, N, Hkv, D, page, kind):
    rng = np.random.default_rng(layers + 10 * N)
    base = rng.integers(1, 90, B).astype(np.int32)
    base[0] = 1
    W = -(-(int(base.max()) + N) // page)
    n_pages = B * W + 2
    table = rng.permutation(n_pages)[: B * W].reshape(B, W).astype(np.int32)
    exps = rng.integers(-4, 5, (layers, 2)).astype(np.int32)
    before = np.stack([random_pages(rng, n_pages, Hkv, page, D) for _ in range(layers)])
    pages = cuda(before)
    nk, nv = values(rng, layers, B, N, Hkv, D), values(rng, layers, B, N, Hkv, D)
    acc = rng.integers(0, min(N, 12), B).astype(np.int32)
    path = np.full((B, 13), -7, np.int32)
    for b in range(B):
        path[b, : acc[b] + 1] = [0, *rng.integers(1, N, acc[b])] if N > 1 else [0]
    args = {"path": (cuda(acc), cuda(path)), "chain": (cuda(acc), None), "all": (None, None)}[kind]
    ws = sv.alloc_workspace(sv.SPEC_MODE_KV4, B, N, 1, sv.SPEC_DTYPE_BF16)
    n = sv.kv4_commit_path(pages, cuda(table), nk, nv, cuda(base), *args, kv_exp=cuda(exps), workspace=ws)
    nodes = [path[b, : acc[b] + 1] if kind == "path" else np.arange((acc[b] if kind == "chain" else N - 1) + 1)
             for b in range(B)]
    assert n.tolist() == [int(base[b]) - 1 + len(nodes[b]) for b in range(B)] and flags_of(ws) == 0
    L = W * page
    k, v = sv.kv4_read(pages, cuda(table), n, L, D, kv_exp=cuda(exps), workspace=ws)
    assert flags_of(ws) == 0
    raw = pages.cpu().numpy()
    touched = np.zeros_like(raw, bool).reshape(layers, n_pages, Hkv, page // 16, 2, 9 * D)
    for layer in range(layers):
        for b in range(B):
            start = int(base[b]) - 1
            old = ref.unpack(before[layer], table[b], start, page, D, exps[layer])
            for got, x, o, e in ((k, nk, old[0], exps[layer, 0]), (v, nv, old[1], exps[layer, 1])):
                got = host(got[layer, b])
                want, _ = ref.rounded(host(x[layer, b])[nodes[b]], int(e))
                assert np.array_equal(got[:start], o)
                assert np.array_equal(got[start: start + len(nodes[b])], want)
                assert (got[start + len(nodes[b]):] == 0).all()  # (left as the call found it)
            for t in range(start, start + len(nodes[b])):
                s = t % page
                grp = touched[layer, table[b, t // page], :, s // 16]
                grp[:, :, (s % 16) * (D // 2): (s % 16 + 1) * (D // 2)] = True
                grp[:, :, 8 * D + (s % 16) * (D // 16): 8 * D + (s % 16 + 1) * (D // 16)] = True
    same = ~touched.reshape(raw.shape)
    assert np.array_equal(raw[same], before[same])


def test_rounding_errors_of_the_format():
    """An element of a block is off by at most half a step of its code, 2^-2 of the
    larger of itself and the smallest step, where the scale is a normal e4m3: the
    scale's own rounding, 2^-4, may also cut the largest at 6 (1 + 2^-4) of it."""
    rng = np.random.default_rng(3)
    x = bf16(rng, 1, 1, 64, 4, 128)
    pages, table = sv.alloc_kv4_pages(1, 1, 4, 64, 128), cuda(np.zeros((1, 1), np.int32))
    n = sv.kv4_commit_path(pages, table, x, x, cuda(np.ones(1, np.int32)))
    k, v = sv.kv4_read(pages, table, n, 64, 128)
    assert torch.equal(k, v)
    y, z = host(x).reshape(-1, 16), host(k).reshape(-1, 16)
    _, s = ref.rounded(y)
    step = ref.SCALES[s][..., 0:1] if s.ndim > 1 else ref.SCALES[s][:, None]
    inside = np.abs(y) <= 6 * step
    bound = np.maximum(np.abs(y) / 4, step / 4)
    assert (np.abs(y - z)[inside] <= bound[inside]).all()
    assert (np.abs(y) <= 6 * step * (1 + 2.0 ** -4) / (1 - 2.0 ** -4)).all()
    assert (np.abs(z)[~inside] == (6 * step * np.ones_like(y))[~inside]).all()


@pytest.mark.parametrize("e", [0, -20, 33])
def test_commit_on_the_borders_of_codes_and_scales(e):
    """Every bf16 magnitude of 25 binades as a block's largest, with the seven borders
    of its codes and a bf16 neighbour of each beside it: bit by bit what exact
    arithmetic gives.  (The 25 binades hold all scales, those below 2^-6 and 448 too.)"""
    a = np.arange(115 << 7, 140 << 7, dtype=np.uint32)  # bf16 bits of 2^-12 .. 2^13
    largest = (a << 16).view(np.float32).astype(np.float64)
    _, s = ref.rounded(np.repeat(largest[:, None], 16, 1))
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * ref.SCALES[s].reshape(-1, 1)
    exact = torch.tensor(borders).to(torch.bfloat16)
    assert (exact.double().numpy() == borders).all()  # (7 bits at most)
    bits = exact.view(torch.int16).numpy().astype(np.int32)
    beside = np.maximum(bits + np.where(np.arange(a.size)[:, None] % 2, 1, -1), 0)
    x = np.concatenate([a[:, None], bits, beside, np.zeros((a.size, 1))], 1).astype(np.int64)
    x = np.where(x > a[:, None], a[:, None], x)  # (none beyond the largest)
    x |= np.random.default_rng(5).integers(0, 2, x.shape) << 15
    x = (x - (x >> 15 << 16)).astype(np.int16).reshape(2, 1, 1, 200, 2, 64)
    k, v = (torch.from_numpy(y).cuda().view(torch.bfloat16) * 2.0 ** e for y in x)
    pages, table = sv.alloc_kv4_pages(1, 4, 2, 64, 64), cuda(np.arange(4, dtype=np.int32)[None])
    exps = cuda(np.full((1, 2), e, np.int32))
    n = sv.kv4_commit_path(pages, table, k, v, cuda(np.ones(1, np.int32)), kv_exp=exps)
    for got, y in zip(sv.kv4_read(pages, table, n, 200, 64, kv_exp=exps), (k, v)):
        want, _ = ref.rounded(host(y), e)
        assert np.array_equal(host(got), want)


def test_commit_of_malformed_sequences():
    """They are left as they were, with the flag of what is wrong; the others are
    written."""
    rng = np.random.default_rng(5)
    B, N, page, D, W = 9, 6, 16, 64, 3
    table = np.arange(B * W).reshape(B, W).astype(np.int32)
    base = np.full(B, 14, np.int32)
    acc = np.full(B, 3, np.int32)
    path = np.tile(np.array([0, 1, 4, 5], np.int32), (B, 1))
    base[0] = 0                    # no root
    acc[1] = 4                     # longer than max_depth
    acc[2] = -1
    path[3, 0] = 1                 # does not start at the root
    path[4, 2] = 6                 # no such node
    path[5, 1] = 0
    table[6, 1] = -1               # positions 13..16: pages 0 and 1
    base[7] = W * page - 1         # beyond the table
    before = np.stack([random_pages(rng, B * W, 2, page, D)])
    pages = cuda(before)
    nk, nv = bf16(rng, 1, B, N, 2, D), bf16(rng, 1, B, N, 2, D)
    ws = sv.alloc_workspace(sv.SPEC_MODE_KV4, B, N, 1, sv.SPEC_DTYPE_BF16)
    n = sv.kv4_commit_path(pages, cuda(table), nk, nv, cuda(base), cuda(acc), cuda(path), workspace=ws)
    assert n.tolist() == [max(int(x) - 1, 0) for x in base[:8]] + [17]
    assert flags_of(ws) == sv.SPEC_FLAG_BAD_PATH | sv.SPEC_FLAG_BAD_PAGE
    raw = pages.cpu().numpy()
    assert np.array_equal(raw[0, : 8 * W], before[0, : 8 * W]) and not np.array_equal(raw[0, 8 * W:], before[0, 8 * W:])
    # one at a time, each its own flag
    for b, flag in ((0, 32), (1, 32), (2, 32), (3, 32), (4, 32), (5, 32), (6, 128), (7, 128)):
        one = slice(b, b + 1)
        sv.kv4_commit_path(pages, cuda(table[one]), nk[:, one].contiguous(), nv[:, one].contiguous(), cuda(base[one]),
                           cuda(acc[one]), cuda(path[one]), workspace=ws)
        assert flags_of(ws) == flag, b


def test_read_lengths_pages_and_strides():
    rng = np.random.default_rng(6)
    B, page, D, Hkv, W, L = 4, 16, 128, 2, 3, 40
    table = np.arange(B * W).reshape(B, W).astype(np.int32)
    table[1, 1] = -3
    raw = np.stack([random_pages(rng, B * W, Hkv, page, D) for _ in range(2)])
    length = np.array([0, 40, -4, 99], np.int32)
    big = torch.full((2, B + 1, L + 3, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = big[:, :B, :L].clone(memory_format=torch.preserve_format), None
    k = big[:, :B, :L]
    vb = big.clone()
    v = vb[:, :B, :L]
    ws = sv.alloc_workspace(sv.SPEC_MODE_KV4, B, 1, 1, sv.SPEC_DTYPE_BF16)
    sv.spec_kv4_read(cuda(raw), cuda(table), cuda(length), k, v, ws)
    assert flags_of(ws) == sv.SPEC_FLAG_BAD_PATH | sv.SPEC_FLAG_BAD_PAGE
    for layer in range(2):
        for b, n in ((0, 0), (1, 40), (2, 0), (3, 40)):
            want = ref.unpack(raw[layer], table[b], n, page, D)
            for got, w in ((k, want[0]), (v, want[1])):
                g = host(got[layer, b])
                assert np.array_equal(g[:n], np.nan_to_num(w)) and (g[n:] == 7).all()
    assert (big[:, B] == 7).all() and (big[:, :, L:] == 7).all()


@pytest.mark.parametrize("first,gap,D", [(0, 0, 64), (8, 0, 64), (0, 8, 128), (16, 16, 64), (8, 24, 128)])
def test_read_into_outputs_of_every_alignment(first, gap, D):
    """Outputs that begin at, and sequences that lie apart by, odd multiples of 16
    bytes and multiples of 32: one result, and nothing beside it is written."""
    rng = np.random.default_rng(7)
    layers, B, page, Hkv, W, L = 2, 3, 16, 3, 2, 27
    table = rng.permutation(B * W).reshape(B, W).astype(np.int32)
    raw = np.stack([random_pages(rng, B * W, Hkv, page, D) for _ in range(layers)])
    row = L * Hkv * D
    flat = [torch.full((layers * B * (row + gap) + 64,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (x[first:].as_strided((layers, B, L, Hkv, D), (B * (row + gap), row + gap, Hkv * D, D, 1), x[first:].storage_offset())
            for x in flat)
    ws = sv.alloc_workspace(sv.SPEC_MODE_KV4, B, 1, 1, sv.SPEC_DTYPE_BF16)
    sv.spec_kv4_read(cuda(raw), cuda(table), cuda(np.array([L, 5, L - 1], np.int32)), k, v, ws)
    assert flags_of(ws) == 0
    for layer in range(layers):
        for b, n in ((0, L), (1, 5), (2, L - 1)):
            for got, w in zip((k, v), ref.unpack(raw[layer], table[b], n, page, D)):
                g = host(got[layer, b])
                assert np.array_equal(g[:n], w) and (g[n:] == 7).all()
    for x, y in zip(flat, (k, v)):
        y.fill_(7.0)
        assert (x == 7).all()


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------

def grid_values(rng, *shape):
    """Values that the format holds exactly, with a scale of 1: a 6 in each 16."""
    x = rng.choice(np.concatenate([ref.CODES, -ref.CODES]), shape)
    x.reshape(-1, 16)[:, 5] = 6.0
    return torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()


def test_rotation_to_nodes_equals_the_one_into_a_cache():
    rng = np.random.default_rng(8)
    B, N, Hq, Hkv, D = 3, 9, 8, 2, 128
    qkv = bf16(rng, B, N, Hq + 2 * Hkv, D)
    w = bf16(rng, D)
    freq = (10000.0 ** (-torch.arange(0, 96, 2) / 96)).float().cuda()
    base = np.array([5, 1, 30], np.int32)
    depth = cuda(rng.integers(0, 5, (B, N)).astype(np.int32))
    kc, vc = (torch.zeros(B, 64, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for inter in (False, True):
        q = sv.tree_qkv_rope(qkv, w, w, 1e-6, freq, cuda(base), depth, kc, vc, 7, inter)
        q2, k2, v2 = sv.tree_qkv_rope_nodes(qkv, Hkv, w, w, 1e-6, freq, cuda(base), depth, 7, inter)
        assert torch.equal(q, q2)
        for b in range(B):
            at = slice(int(base[b]) - 1, int(base[b]) - 1 + N)
            assert torch.equal(kc[b, at], k2[b]) and torch.equal(vc[b, at], v2[b])
    ws = sv.alloc_workspace(sv.SPEC_MODE_TREE_QKV, B, N, 1, sv.SPEC_DTYPE_BF16)
    base[1] = 0
    q3, k3, v3 = sv.tree_qkv_rope_nodes(qkv, Hkv, w, w, 1e-6, freq, cuda(base), depth, 7, True, ws)
    assert flags_of(ws) == sv.SPEC_FLAG_BAD_PATH and (q3[1] == 0).all()
    assert torch.equal(q3[0], q2[0]) and torch.equal(k3[2], k2[2])


@pytest.mark.parametrize("N,Hq", [(5, 8), (40, 8)])
def test_steps_of_tree_decoding_against_the_bf16_cache(N, Hq):
    """Drafts, attention, walk, commit and growth, some steps long, over pages that
    hold the values exactly: every step's attention against 64 bits, and the
    4-bit cache against the bf16 one that spec_kv_commit_path keeps."""
    rng = np.random.default_rng(N)
    B, Hkv, D, page, V, L, W = 3, 2, 64, 16, 97, 400, 25
    n_pages = 60
    pages = sv.alloc_kv4_pages(1, n_pages, Hkv, page, D)
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(B, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for step in range(6):
        parents = np.stack([[-1] + [int(rng.integers(max(0, v - 4), v)) for v in range(1, N)] for _ in range(B)]).astype(np.int32)
        mask, depth = sv.tree_attention_mask(cuda(parents))
        base = length + 1
        kv = [grid_values(rng, B, N, Hkv, D) for _ in range(2)]
        qkv = torch.cat([bf16(rng, B, N, Hq, D), *kv], 2).contiguous()
        # both caches
        q = sv.tree_qkv_rope(qkv, None, None, 0.0, None, base, depth, kc, vc)
        q2, nk, nv = sv.tree_qkv_rope_nodes(qkv, Hkv, None, None, 0.0, None, base, depth)
        assert torch.equal(q, q2)
        a = sv.tree_attention(q, kc, vc, mask, base)
        b = sv.tree_attention_kv4(q2, pages[0], table, nk, nv, mask, base)
        # weights of 2^-9 (bf16) and 2^-11, an output's 2^-8 twice: all of |v| <= 6
        assert (a[0].float() - b[0].float()).abs().max() <= 6 * (2.0 ** -7 + 2 * 2.0 ** -9 + 2 * 2.0 ** -11)
        assert torch.allclose(a[1], b[1], atol=1e-3, rtol=1e-5)
        logits = bf16(rng, B, N, V, scale=3.0)
        tokens = torch.randint(0, 12, (B, N), dtype=torch.int32, device="cuda")
        logits[..., :12] += 6
        r = sv.verify_tree_sample(logits, tokens, cuda(parents), torch.rand(B, 9, device="cuda"), 1.0, 8)
        # pages for what is accepted, then the commits
        need = length + r["accepted_len"] + 1
        table, length, used = sv.kv_pages_fork(pages, table, length, None, need, page)
        new = sv.kv4_commit_path(pages, table, nk[None], nv[None], base, r["accepted_len"], r["path_nodes"])
        cache = torch.stack([kc, vc])
        new_len = torch.empty_like(new)
        sv.spec_kv_commit_path(cache, base, r["accepted_len"], r["path_nodes"], N, new_len,
                               sv.alloc_workspace(sv.SPEC_MODE_KV_COMMIT, B, N, 1, 0))
        kc, vc = cache[0].contiguous(), cache[1].contiguous()
        assert torch.equal(new, new_len) and torch.equal(new, need)
        length = new
        k, v = sv.kv4_read(pages, table, length, L, D)
        for s in range(B):
            n = int(length[s])
            assert torch.equal(k[0, s, :n], kc[s, :n]) and torch.equal(v[0, s, :n], vc[s, :n])
        assert int(used) == sum(-(-int(n) // page) for n in length)


def test_steps_of_beam_decoding():
    """Prompt, then beams: selection, fork of the pages by its parents, commit and
    attention.  Each beam's cache has to hold its own history."""
    rng = np.random.default_rng(11)
    K, Hkv, Hq, D, page, V, W, layers = 4, 2, 8, 64, 16, 50, 8, 2
    pages = sv.alloc_kv4_pages(layers, 40, Hkv, page, D)
    prompt = 21
    table = torch.full((1, W), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, length, used = sv.kv_pages_fork(pages, table, zero, None, zero + prompt, page)
    pk, pv = grid_values(rng, layers, 1, prompt, Hkv, D), grid_values(rng, layers, 1, prompt, Hkv, D)
    length = sv.kv4_commit_path(pages, table, pk, pv, zero + 1)
    history = [(pk[:, 0], pv[:, 0])]
    scores = torch.tensor([[0.0] + [-float("inf")] * (K - 1)], device="cuda")
    finished = torch.zeros(1, K, dtype=torch.int32, device="cuda")
    table = torch.cat([table] + [torch.full_like(table, -1)] * (K - 1)).contiguous()
    length = torch.cat([length] + [torch.zeros_like(length)] * (K - 1)).contiguous()
    history += [None] * (K - 1)
    for step in range(30):
        logits = bf16(rng, 1, K, V, scale=2.0)
        r = sv.beam_select(logits, scores, K, finished, eos=3)
        parents = r["parents"].view(-1)
        grow = torch.where(parents >= 0, length[parents.clamp(min=0).long()] + 1, 0).int()
        table, length, used = sv.kv_pages_fork(pages, table, length, parents, grow, page)
        nk, nv = grid_values(rng, layers, K, 1, Hkv, D), grid_values(rng, layers, K, 1, Hkv, D)
        if step % 7 == 3:
            table, n = sv.kv_pages_compact(pages, table)
            assert int(n) == int(used) and int(table.max()) < int(n)
        length = sv.kv4_commit_path(pages, table, nk, nv, length + 1)
        history = [(torch.cat([history[p][0], nk[:, j]], 1), torch.cat([history[p][1], nv[:, j]], 1))
                   for j, p in enumerate(parents.tolist())]
        scores, finished = r["scores"], r["finished"]
        k, v = sv.kv4_read(pages, table, length, W * page, D)
        q = bf16(rng, K, 1, Hq, D)
        out, lse = sv.tree_attention_kv4(q, pages[0], table, nk[0], nv[0], None, length, scale=0.1)
        for j in range(K):
            n = int(length[j])
            assert n == prompt + step + 1
            assert torch.equal(k[:, j, :n], history[j][0]) and torch.equal(v[:, j, :n], history[j][1])
            want, wl, mass, amp = ref.attention(host(q[j]), host(history[j][0][0]), host(history[j][1][0]),
                                                np.ones((1, n), bool), 0.1)
            ds = D * 2.0 ** -23 * amp + 4e-5
            assert (np.abs(host(lse[j]) - wl) <= ds + 2.0 ** -22 * np.abs(wl)).all()
            assert (np.abs(host(out[j]) - want) <= 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -11 + ds[..., None]) * mass).all()
        live = {int(x) for x in table.view(-1) if x >= 0}
        assert int(used) == len(live)
