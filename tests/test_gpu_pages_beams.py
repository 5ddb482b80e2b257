"""Forks and compaction of pages, and beam selection, on the GPU against plain
implementations."""
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


def tables(rng, B, W, page, n_pages, share=0.5):
    """Sequences that share leading pages with an earlier one, some of odd lengths."""
    length = rng.integers(0, W * page + 1, B).astype(np.int32)
    ids = rng.permutation(n_pages).tolist()
    table = np.full((B, W), -1, np.int32)
    for b in range(B):
        n, s = -(-int(length[b]) // page), 0
        if b and rng.random() < share:
            o = int(rng.integers(0, b))
            s = int(rng.integers(0, min(length[b] // page, length[o] // page) + 1))
            table[b, :s] = table[o, :s]
        for i in range(s, n):
            if not ids:
                length[b] = i * page
                break
            table[b, i] = ids.pop()
    return table, length


def check_fork(rng, table, length, parent, need, page, n_pages, planes=3, words=4, stream=None):
    pages = torch.randint(0, 1 << 30, (planes, n_pages, words), dtype=torch.int32, device="cuda",
                          generator=torch.Generator("cuda").manual_seed(int(rng.integers(1 << 30))))
    old = pages.clone()
    ws = sv.alloc_kv_pages_workspace(pages, len(parent))
    new, ln, used = sv.kv_pages_fork(pages, cuda(table), cuda(length), cuda(parent), cuda(need), page, ws, stream)
    torch.cuda.synchronize()
    want, wl, wu, copies = ref.fork(table, length, parent, need, page, n_pages)
    assert np.array_equal(new.cpu().numpy(), want)
    assert np.array_equal(ln.cpu().numpy(), wl) and int(used) == wu
    for a, b in copies:
        old[:, b] = old[:, a]
    assert torch.equal(pages, old)
    return sv.spec_verify_read_flags(ws), want, wl


@pytest.mark.parametrize("B,B2,W,page,n_pages", [
    (1, 1, 1, 16, 1), (1, 4, 5, 16, 40), (8, 8, 7, 32, 90), (5, 17, 6, 1, 150), (64, 64, 18, 64, 1400),
    (3, 512, 4, 3, 2500), (200, 300, 9, 128, 3000), (3, 2, 2, 7, 32),
    (600, 600, 5, 16, 4000),        # more sequences than the small plan takes
    (10, 12, 6, 16, 40000),         # more pages
    (20, 9, 5000, 16, 60000),       # more table entries
    (4, 1500, 6, 16, 9001), (900, 2100, 3, 16, 33000),
])
def test_fork(B, B2, W, page, n_pages):
    rng = np.random.default_rng(B + B2 + W)
    table, length = tables(rng, B, W, page, n_pages)
    parent = rng.integers(-1, B, B2).astype(np.int32)
    need = np.where(parent >= 0, np.minimum(length[parent] + rng.integers(0, 2 * page, B2), W * page), 0).astype(np.int32)
    flags, new, ln = check_fork(rng, table, length, parent, need, page, n_pages)
    full = (new.reshape(-1) >= 0).sum()
    assert flags in (0, sv.SPEC_FLAG_NO_PAGE) and full >= 0
    if flags == 0:
        # every position to come stands in a page that its sequence alone holds
        held = {}
        for j in range(B2):
            for i, x in enumerate(new[j]):
                if x >= 0:
                    held.setdefault(int(x), []).append((j, i))
        for x, who in held.items():
            for j, i in who:
                if (i + 1) * page > ln[j]:
                    assert len(who) == 1


def test_fork_growth_alone_and_empty():
    rng = np.random.default_rng(2)
    table, length = tables(rng, 6, 5, 16, 60)
    pages = torch.zeros(1, 60, 4, dtype=torch.int32, device="cuda")
    need = np.minimum(length + 20, 80).astype(np.int32)
    got = sv.kv_pages_fork(pages, cuda(table), cuda(length), None, cuda(need), 16)
    want = ref.fork(table, length, np.arange(6), need, 16, 60)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and int(got[2]) == want[2]
    none = sv.kv_pages_fork(pages, cuda(table), cuda(length), cuda(np.full(6, -1, np.int32)), None, 16)
    assert (none[0] == -1).all() and (none[1] == 0).all() and int(none[2]) == 0


@pytest.mark.parametrize("n_pages", [60, 40000])
def test_fork_of_bad_data(n_pages):
    """Parents, lengths, needs and entries outside their ranges: flagged, the rest
    as the definition has it."""
    rng = np.random.default_rng(4)
    page, W = 16, 4
    table, length = tables(rng, 8, W, page, 60, share=0.3)
    length[:] = [20, 33, 64, 5, 16, 40, 17, 1]
    table[:] = np.arange(32).reshape(8, 4)
    table[0, 1] = -1          # an unfinished page that is none: a fresh one, no copy
    table[1, 0] = n_pages     # a full page that is none
    cases = [
        ([0, 1, 2], [40, 40, 64], length, sv.SPEC_FLAG_BAD_PAGE),
        ([8, -2, 3], [0, 9, 40], length, sv.SPEC_FLAG_BAD_PARENT),
        ([2, 3], [9999, 5], length, sv.SPEC_FLAG_BAD_PATH),
        ([4, 5], [16, 40], np.array([20, 33, 64, 5, -1, 65, 17, 1], np.int32), sv.SPEC_FLAG_BAD_PATH),
    ]
    for parent, need, ln, flag in cases:
        got, _, _ = check_fork(rng, table, ln, np.array(parent, np.int32), np.array(need, np.int32), page, n_pages)
        assert got == flag
    small = 9
    t = np.full((2, W), -1, np.int32)
    t[0, :2], t[1, 0] = [3, 5], 7
    got, new, _ = check_fork(rng, t, np.array([20, 4], np.int32), np.array([0, 0, 1, 1], np.int32),
                             np.array([64, 64, 64, 64], np.int32), page, small)
    assert got == sv.SPEC_FLAG_NO_PAGE and (new == -1).any()


@pytest.mark.parametrize("B,W,n_pages", [(1, 1, 1), (3, 5, 40), (24, 24, 900), (8, 7, 33000), (700, 100, 71000), (2, 3, 1500)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(B, W, n_pages, in_place):
    rng = np.random.default_rng(B + W)
    table, _ = tables(rng, B, W, 16, n_pages)
    table[rng.random(table.shape) < 0.1] = -1
    pages = torch.randint(0, 255, (2, n_pages, 32), dtype=torch.uint8, device="cuda")
    old = pages.clone()
    want, n, moves = ref.compact(table, n_pages)
    ws = sv.alloc_kv_pages_workspace(pages, B)
    dev = cuda(table)
    new = dev if in_place else torch.empty_like(dev)
    used = torch.empty(1, dtype=torch.int32, device="cuda")
    sv.spec_kv_pages_compact(pages, dev, new, used, ws)
    assert np.array_equal(new.cpu().numpy(), want) and int(used) == n
    for a, b in moves:
        old[:, b] = old[:, a]
    assert torch.equal(pages, old) and sv.spec_verify_read_flags(ws) == 0


def test_compact_of_bad_entries():
    pages = torch.arange(6 * 16, dtype=torch.int32, device="cuda").view(1, 6, 16)
    ws = sv.alloc_kv_pages_workspace(pages, 2)
    new, used = sv.kv_pages_compact(pages, cuda(np.array([[5, -7, 6], [5, 4, -1]], np.int32)), ws)
    assert new.tolist() == [[1, -1, -1], [1, 0, -1]] and int(used) == 2
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PAGE
    assert pages[0, 0, 0] == 4 * 16 and pages[0, 1, 0] == 5 * 16


def test_pages_on_another_stream_captured_and_in_a_tight_workspace():
    rng = np.random.default_rng(9)
    table, length = tables(rng, 12, 6, 16, 100)
    parent = rng.integers(0, 12, 12).astype(np.int32)
    need = np.minimum(length[parent] + 5, 96).astype(np.int32)
    check_fork(rng, table, length, parent, need, 16, 100, stream=torch.cuda.Stream())
    n = sv.spec_kv_pages_workspace_bytes(100, 12)
    buf = torch.full((n + 4096,), 0xEE, dtype=torch.uint8, device="cuda")
    buf[:4] = 0
    pages = torch.randint(0, 99, (2, 100, 8), dtype=torch.int32, device="cuda")
    t, ln, par, nd = cuda(table), cuda(length), cuda(parent), cuda(need)
    out = (torch.empty(12, 6, dtype=torch.int32, device="cuda"), torch.empty(12, dtype=torch.int32, device="cuda"),
           torch.empty(1, dtype=torch.int32, device="cuda"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_kv_pages_fork(pages, t, ln, par, nd, 16, *out, buf[:n])
        sv.spec_kv_pages_compact(pages, out[0], out[0], out[2], buf[:n])
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        a, b = tables(r, 12, 6, 16, 100)
        t.copy_(cuda(a)), ln.copy_(cuda(b)), nd.copy_(cuda(np.minimum(b[parent] + 5, 96).astype(np.int32)))
        g.replay()
        f = ref.fork(a, b, parent, np.minimum(b[parent] + 5, 96), 16, 100)
        want, used, _ = ref.compact(f[0], 100)
        assert np.array_equal(out[0].cpu().numpy(), want) and int(out[2]) == used
    assert (buf[n:] == 0xEE).all()


def test_pages_of_a_pool_beyond_32_bit_offsets():
    pages = torch.empty(2, 5, 500_000_000 // 4 * 2, dtype=torch.int16, device="cuda")
    for i in range(5):
        pages[:, i].fill_(i)
    table = cuda(np.array([[4, 3]], np.int32))
    new, _, used = sv.kv_pages_fork(pages, table, cuda(np.array([20], np.int32)), cuda(np.array([0, 0], np.int32)), None, 16)
    assert new.tolist() == [[4, 3], [4, 0]] and int(used) == 3
    assert (pages[:, 0] == 3).all() and (pages[:, 3] == 3).all() and (pages[:, 1] == 1).all()
    new, used = sv.kv_pages_compact(pages, new)
    assert new.tolist() == [[2, 1], [2, 0]] and (pages[:, 2] == 4).all() and (pages[:, 1] == 3).all()


# ---------------------------------------------------------------------------
# beams
# ---------------------------------------------------------------------------

def check_beams(logits, scores, M, finished=None, eos=-1, T=1.0, workspace=None, stream=None):
    """Totals are off by less than 2^-19 (1 + |z / T|), as documented, and half a
    step of float32; places may differ where two totals lie closer than that."""
    got = {k: v.cpu().numpy() for k, v in sv.beam_select(
        logits, cuda(scores), M, None if finished is None else cuda(finished), eos, T, workspace, stream).items()}
    z = logits.double().cpu().numpy()
    (s, p, t, f), every = ref.beams(z, scores, finished, eos, T, M)
    big = np.abs(np.where(np.isfinite(z), z, 0)).max() / T
    tol = 2.0 ** -19 * (1 + big)
    for b in range(len(s)):
        gaps = -np.diff(np.array(every[b][: M + 1])) if len(every[b]) > 1 else np.array([1.0])
        exact = (gaps > 2 * tol) | (gaps == 0)
        ok = np.isfinite(s[b])
        assert np.array_equal(ok, np.isfinite(got["scores"][b]))
        assert (np.abs(got["scores"][b][ok] - s[b][ok]) <= tol + 2.0 ** -24 * np.abs(s[b][ok])).all()
        if exact.all():
            assert np.array_equal(got["parents"][b], p[b]) and np.array_equal(got["tokens"][b], t[b])
            assert np.array_equal(got["finished"][b], f[b])
        else:
            assert len({(x, y) for x, y in zip(got["parents"][b][ok], got["tokens"][b][ok])}) == ok.sum()
    return got


def draws(rng, B, K, V, dtype, scale=2.0):
    z = torch.from_numpy((rng.standard_normal((B, K, V)) * scale).astype(np.float32))
    return z.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


@pytest.mark.parametrize("B,K,V,M", [
    (1, 1, 1, 1), (2, 3, 5, 4), (1, 4, 1000, 4), (3, 5, 32003, 8), (2, 8, 16384, 16), (1, 64, 700, 16), (5, 2, 128256, 6),
    (2, 12, 8193, 3), (1, 2, 400000, 16), (1, 17, 40000, 9),
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beams(B, K, V, M, dtype):
    rng = np.random.default_rng(V + K)
    scores = (-3 * rng.random((B, K)) - 1).astype(np.float32)
    finished = (rng.random((B, K)) < 0.2).astype(np.int32)
    z = draws(rng, B, K, V, dtype)
    check_beams(z, scores, M)
    check_beams(z, scores, M, finished, eos=min(2, V - 1), T=0.7)


@pytest.mark.parametrize("V", [1024, 5003, 70000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beams_ties(V, dtype):
    """Few distinct logits: the lowest beams and tokens win; equal rows tie, whatever
    memory they start at and however they are cut."""
    rng = np.random.default_rng(V)
    z = torch.from_numpy(rng.integers(0, 3, (4, 6, V)).astype(np.float32))
    z[1] = z[1, 0]
    z[2] = 0.5
    z[3, :, 17:] = -float("inf")
    z = z.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    for M in (1, 7, 16):
        got = check_beams(z, np.zeros((4, 6), np.float32), M)
        assert got["tokens"][2].tolist() == list(range(M)) and (got["parents"][2] == 12).all()
        first = np.flatnonzero(z[1, 0].float().cpu().numpy() == 2)
        assert got["tokens"][1].tolist() == first[:M].tolist() and (got["parents"][1] == 6).all()


def test_beams_many_large_logits_in_one_run():
    """More candidates than lanes in one run, and the best ones elsewhere."""
    rng = np.random.default_rng(1)
    z = draws(rng, 2, 3, 50000, "f32", 1.0)
    z[:, :, 1000:1300] += 20
    z[0, 1, 49999] = 40
    z[1, 2, 0] = 39
    check_beams(z, -rng.random((2, 3)).astype(np.float32), 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [640, 3001])
def test_beams_without_candidates(dtype, V):
    rng = np.random.default_rng(V)
    z = draws(rng, 5, 3, V, dtype)
    scores = -rng.random((5, 3)).astype(np.float32)
    scores[0] = -np.inf                   # no beam
    scores[1, 1:] = -np.inf               # the first step
    z[2, :, 1:] = -float("inf")           # one token a beam
    z[3, 0] = -float("inf")               # a row of none
    scores[4, 0] = np.nan
    fin = np.zeros((5, 3), np.int32)
    fin[1, 2] = 1                         # finished, with a score of -inf
    fin[4, 2] = 1
    got = check_beams(z, scores, 5, fin, eos=4)
    assert (got["parents"][0] == -1).all() and (got["tokens"][0] == -1).all() and (got["finished"][0] == 1).all()
    assert (got["tokens"][2][:3] == 0).all() and (got["parents"][2][3:] == -1).all()


def test_beams_on_another_stream_captured_and_in_a_tight_workspace():
    rng = np.random.default_rng(3)
    z = draws(rng, 3, 4, 20000, "bf16")
    scores = -rng.random((3, 4)).astype(np.float32)
    n = sv.spec_beam_select_workspace_bytes(3, 4, 20000, 4, sv.SPEC_DTYPE_BF16)
    buf = torch.full((n + 4096,), 0xEE, dtype=torch.uint8, device="cuda")
    buf[:4] = 0
    want = check_beams(z, scores, 4, workspace=buf[:n], stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert (buf[n:] == 0xEE).all()
    dev = cuda(scores)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.empty(3, 4, device="cuda")] + [torch.empty(3, 4, **i32) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_beam_select(z, dev, None, -1, 1.0, *out, buf[:n])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out[1].cpu().numpy(), want["parents"]) and np.array_equal(out[2].cpu().numpy(), want["tokens"])
        assert np.array_equal(out[0].cpu().numpy(), want["scores"])
        z.copy_(draws(rng, 3, 4, 20000, "bf16"))
        want = check_beams(z, scores, 4)
