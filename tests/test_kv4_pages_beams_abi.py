"""CPU checks of the calls on the 4-bit cache, on pages and on beams: workspace
sizes and refusals (every call below fails validation or is the B = 0 no-op,
before any CUDA call), the wrappers' refusals that need no GPU, and the
references that the GPU tests compare with."""
import numpy as np
import pytest

import kv4_reference as ref
import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build
from test_tree_forward_abi import ALIGN, FAKE, INVALID, OK, WORKSPACE, caller


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return sv.load_library()


def test_workspace_sizes(lib):
    assert sv.spec_verify_workspace_bytes(sv.SPEC_MODE_KV4, 4, 60, 1, sv.SPEC_DTYPE_BF16) == 256
    at = sv.spec_tree_attention_kv4_workspace_bytes
    for shape in ((64, 1, 32, 8, 128), (16, 60, 32, 8, 128), (1, 1, 1, 1, 64)):
        assert at(*shape) > 0 and at(*shape) % 256 == 0
    assert at(64, 1, 32, 8, 128) < 8 << 20
    for bad in ((-1, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 4097, 8, 8, 64), (1, 1, 30, 8, 64), (1, 1, 8, 0, 64),
                (1, 1, 129, 1, 64), (1, 1, 8, 8, 96), (1 << 24, 4096, 8, 8, 64)):
        assert at(*bad) == 0, bad
    pg = sv.spec_kv_pages_workspace_bytes
    assert 0 < pg(100, 4) < pg(100000, 4) and pg(100, 4) % 256 == 0
    assert pg(0, 1) == 0 and pg((1 << 24) + 1, 1) == 0 and pg(10, -1) == 0 and pg(10, (1 << 20) + 1) == 0
    bm = sv.spec_beam_select_workspace_bytes
    assert 0 < bm(1, 4, 128256, 4, 1) < bm(64, 8, 128256, 8, 1)
    for bad in ((-1, 4, 10, 4, 1), (1, 0, 10, 1, 1), (1, 65, 10, 1, 1), (1, 4, 0, 1, 1), (1, 4, 10, 0, 1),
                (1, 4, 10, 17, 1), (1, 4, 10, 4, 2), (1 << 20, 64, 128256, 4, 1)):
        assert bm(*bad) == 0, bad


def test_commit_validation(lib):
    call = caller(lib.spec_kv4_commit_path, pages=FAKE, layers=2, n_pages=9, page=16, Hkv=2, D=64, table=FAKE, W=3,
                  nk=FAKE, nv=FAKE, base=FAKE, acc=FAKE, path=FAKE, md=4, exps=None, B=2, N=8, new=FAKE, ws=FAKE,
                  wsb=256, stream=None)
    for over in (dict(layers=0), dict(n_pages=0), dict(n_pages=1 << 31), dict(page=8), dict(page=48), dict(page=256),
                 dict(Hkv=0), dict(D=96), dict(W=0), dict(W=(1 << 20) + 1), dict(md=-1), dict(md=1025), dict(acc=None),
                 dict(B=-1), dict(N=0), dict(N=65537), dict(B=1 << 26), dict(pages=None), dict(table=None),
                 dict(nk=None), dict(nv=None), dict(base=None), dict(new=None)):
        assert call(**over) == INVALID, over
    for over in (dict(pages=FAKE + 8), dict(nk=FAKE + 8), dict(nv=FAKE + 2), dict(table=FAKE + 2), dict(base=FAKE + 1),
                 dict(acc=FAKE + 2), dict(path=FAKE + 2), dict(exps=FAKE + 2), dict(new=FAKE + 2), dict(ws=FAKE + 128)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE
    assert call(B=0, pages=None, ws=None) == OK


def test_read_validation(lib):
    seq = 40 * 2 * 64 * 2
    call = caller(lib.spec_kv4_read, pages=FAKE, layers=2, n_pages=9, page=16, Hkv=2, D=64, table=FAKE, W=3, len=FAKE,
                  exps=None, B=2, L=40, k=FAKE, v=FAKE, ls=2 * seq, ss=seq, ws=FAKE, wsb=256, stream=None)
    for over in (dict(layers=0), dict(page=17), dict(D=32), dict(B=-1), dict(L=0), dict(ss=seq - 16), dict(ls=2 * seq - 16),
                 dict(ss=1 << 62, ls=1 << 62), dict(pages=None), dict(table=None), dict(len=None), dict(k=None), dict(v=None)):
        assert call(**over) == INVALID, over
    for over in (dict(k=FAKE + 8), dict(v=FAKE + 4), dict(ss=seq + 8, ls=4 * seq), dict(ls=2 * seq + 8), dict(len=FAKE + 2)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=100) == WORKSPACE
    assert call(B=0, k=None) == OK


@pytest.mark.parametrize("N", [1, 60])
def test_attention_validation(lib, N):
    n = sv.spec_tree_attention_kv4_workspace_bytes(2, N, 8, 2, 64)
    call = caller(lib.spec_tree_attention_kv4, q=FAKE, pages=FAKE, n_pages=9, page=16, table=FAKE, W=3, nk=FAKE, nv=FAKE,
                  mask=None, base=FAKE, exps=None, B=2, N=N, Hq=8, Hkv=2, D=64, scale=0.1, out=FAKE, lse=None, ws=FAKE,
                  wsb=n, stream=None)
    inf, nan = float("inf"), float("nan")
    for over in (dict(n_pages=0), dict(page=20), dict(W=0), dict(B=-1), dict(N=0), dict(N=4097), dict(Hq=7), dict(Hkv=0),
                 dict(Hq=258), dict(D=80), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf), dict(scale=nan),
                 dict(scale=1.8e38), dict(q=None), dict(pages=None), dict(table=None), dict(nk=None), dict(nv=None),
                 dict(base=None), dict(out=None)):
        assert call(**over) == INVALID, over
    for over in (dict(q=FAKE + 8), dict(pages=FAKE + 4), dict(nk=FAKE + 2), dict(nv=FAKE + 8), dict(out=FAKE + 2),
                 dict(mask=FAKE + 2), dict(lse=FAKE + 2), dict(exps=FAKE + 1), dict(base=FAKE + 3), dict(ws=FAKE + 64)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=n - 1) == WORKSPACE
    assert call(B=0, q=None, ws=None) == OK


def test_pages_validation(lib):
    n = sv.spec_kv_pages_workspace_bytes(9, 4)
    fork = caller(lib.spec_kv_pages_fork, pages=FAKE, planes=2, ps=9 * 64, n_pages=9, pb=64, page=16, table=FAKE, len=FAKE,
                  B=3, parent=FAKE, need=None, B2=4, W=3, new=FAKE, nl=FAKE, used=FAKE, ws=FAKE, wsb=n, stream=None)
    for over in (dict(planes=0), dict(ps=9 * 64 - 16), dict(n_pages=0), dict(n_pages=(1 << 24) + 1), dict(pb=8), dict(page=0),
                 dict(B=-1), dict(B2=-1), dict(W=0), dict(W=1 << 20, page=1 << 12), dict(parent=None), dict(pages=None),
                 dict(table=None), dict(len=None), dict(new=None), dict(nl=None), dict(used=None), dict(pb=1 << 62),
                 dict(B2=(1 << 20) + 1)):
        assert fork(**over) == INVALID, over
    for over in (dict(pages=FAKE + 8), dict(pb=72, ps=9 * 80), dict(ps=9 * 64 + 8), dict(table=FAKE + 2), dict(len=FAKE + 2),
                 dict(parent=FAKE + 2), dict(need=FAKE + 2), dict(new=FAKE + 2), dict(used=FAKE + 1), dict(ws=FAKE + 8)):
        assert fork(**over) == ALIGN, over
    assert fork(ws=None) == WORKSPACE and fork(wsb=n - 1) == WORKSPACE
    compact = caller(lib.spec_kv_pages_compact, pages=FAKE, planes=2, ps=9 * 64, n_pages=9, pb=64, table=FAKE, B=3, W=3,
                     new=FAKE, used=FAKE, ws=FAKE, wsb=n, stream=None)
    for over in (dict(planes=0), dict(n_pages=-1), dict(W=0), dict(table=None), dict(new=None), dict(used=None)):
        assert compact(**over) == INVALID, over
    assert compact(pages=FAKE + 4) == ALIGN and compact(wsb=10) == WORKSPACE


def test_beam_validation(lib):
    n = sv.spec_beam_select_workspace_bytes(2, 4, 1000, 4, 1)
    call = caller(lib.spec_beam_select, z=FAKE, dtype=1, s=FAKE, fin=None, eos=2, T=1.0, B=2, K=4, V=1000, M=4, os=FAKE,
                  op=FAKE, ot=FAKE, of=FAKE, ws=FAKE, wsb=n, stream=None)
    for over in (dict(dtype=2), dict(eos=-2), dict(eos=1000), dict(T=0.0), dict(T=float("nan")), dict(T=float("inf")),
                 dict(B=-1), dict(K=0), dict(K=65), dict(V=0), dict(V=(1 << 26) + 1), dict(M=0), dict(M=17), dict(z=None),
                 dict(s=None), dict(os=None), dict(op=None), dict(ot=None), dict(of=None), dict(B=1 << 20, V=1 << 26)):
        assert call(**over) == INVALID, over
    for over in (dict(z=FAKE + 1), dict(dtype=0, z=FAKE + 2), dict(s=FAKE + 2), dict(fin=FAKE + 2), dict(op=FAKE + 2),
                 dict(ws=FAKE + 32)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=n - 1) == WORKSPACE
    assert call(B=0, z=None) == OK


def test_outputs_over_inputs(lib):
    far = [FAKE + (i << 30) for i in range(1, 10)]
    call = caller(lib.spec_kv4_commit_path, pages=far[0], layers=2, n_pages=9, page=16, Hkv=2, D=64, table=far[1], W=3,
                  nk=far[2], nv=far[3], base=far[4], acc=far[5], path=far[6], md=4, exps=None, B=2, N=8, new=far[7],
                  ws=far[8], wsb=256, stream=None)
    for over in (far[4], far[4] + 4, far[5], far[6] + 36, far[1] + 20):
        assert call(new=over) == INVALID, over
    for N in (1, 60):
        n = sv.spec_tree_attention_kv4_workspace_bytes(2, N, 8, 2, 64)
        call = caller(lib.spec_tree_attention_kv4, q=far[0], pages=far[1], n_pages=9, page=16, table=far[2], W=3, nk=far[3],
                      nv=far[4], mask=None, base=far[5], exps=None, B=2, N=N, Hq=8, Hkv=2, D=64, scale=0.1, out=far[6],
                      lse=None, ws=far[7], wsb=n, stream=None)
        for over in (far[0], far[0] + 2 * 2 * N * 8 * 64 - 16, far[0] - 2 * 2 * N * 8 * 64 + 16, far[3], far[4]):
            assert call(out=over) == INVALID, over
    n = sv.spec_kv_pages_workspace_bytes(9, 4)
    fork = caller(lib.spec_kv_pages_fork, pages=far[0], planes=2, ps=9 * 64, n_pages=9, pb=64, page=16, table=far[1],
                  len=far[2], B=3, parent=far[3], need=far[4], B2=4, W=3, new=far[5], nl=far[6], used=far[7], ws=far[8],
                  wsb=n, stream=None)
    for over in (dict(new=far[1]), dict(new=far[1] + 32), dict(new=far[2]), dict(nl=far[2]), dict(nl=far[3]),
                 dict(nl=far[4] + 12), dict(used=far[1]), dict(used=far[2] + 8)):
        assert fork(**over) == INVALID, over
    compact = caller(lib.spec_kv_pages_compact, pages=far[0], planes=2, ps=9 * 64, n_pages=9, pb=64, table=far[1], B=3, W=3,
                     new=far[5], used=far[7], ws=far[8], wsb=n, stream=None)
    for over in (dict(new=far[1] + 4), dict(new=far[1] - 4), dict(used=far[1] + 32)):
        assert compact(**over) == INVALID, over
    n = sv.spec_beam_select_workspace_bytes(2, 4, 1000, 4, 1)
    call = caller(lib.spec_beam_select, z=far[0], dtype=1, s=far[1], fin=far[2], eos=2, T=1.0, B=2, K=4, V=1000, M=4,
                  os=far[3], op=far[4], ot=far[5], of=far[6], ws=far[7], wsb=n, stream=None)
    for over in (dict(os=far[1]), dict(op=far[1] + 28), dict(ot=far[2]), dict(of=far[2])):
        assert call(**over) == INVALID, over


def test_rope_nodes_validation(lib):
    call = caller(lib.spec_tree_qkv_rope_nodes, qkv=FAKE, qn=None, kn=None, eps=1e-6, freq=FAKE, rot=64, inter=0, off=0,
                  base=FAKE, depth=None, B=2, N=8, Hq=8, Hkv=2, D=64, q=FAKE, k=FAKE, v=FAKE, ws=FAKE, wsb=256, stream=None)
    for over in (dict(rot=66), dict(rot=3), dict(N=0), dict(Hkv=0), dict(D=32), dict(off=-1), dict(qkv=None), dict(k=None),
                 dict(freq=None), dict(eps=-1.0)):
        assert call(**over) == INVALID, over
    for over in (dict(qkv=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(base=FAKE + 2)):
        assert call(**over) == ALIGN, over
    assert call(wsb=255) == WORKSPACE and call(B=0, q=None) == OK


def test_wrappers_refuse_what_is_not_on_a_gpu():
    import torch
    z = torch.zeros(1, 2, 10)
    pages = torch.zeros(1, 4, 2, 9 * 16 * 64 // 8, dtype=torch.uint8)
    table, one = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    kv, ws = torch.zeros(1, 1, 3, 2, 64, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: sv.spec_beam_select(z, z[0], None, -1, 1.0, z[0], table, table, table, ws),
                 lambda: sv.spec_kv4_commit_path(pages, table, kv, kv, one, None, None, one, ws),
                 lambda: sv.spec_kv4_read(pages, table, one, kv, kv, ws),
                 lambda: sv.spec_tree_attention_kv4(kv[0], pages[0], table, kv[0], kv[0], None, one, 1.0, kv[0], None, ws),
                 lambda: sv.spec_kv_pages_fork(pages, table, one, one, None, 16, table, one, one, ws),
                 lambda: sv.spec_kv_pages_compact(pages, table, table, one, ws)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
    for bad in ((1, 4, 2, 17, 64), (1, 4, 2, 16, 96)):
        with pytest.raises(ValueError):
            sv.alloc_kv4_pages(*bad, device="cpu")
    assert sv.alloc_kv4_pages(2, 3, 4, 32, 128, device="cpu").shape == (2, 3, 4, 9 * 32 * 128 // 8)


def test_reference_rounding_against_brute_force():
    """Scales and codes against all candidates, in fractions of 2^-20."""
    rng = np.random.default_rng(0)
    x = np.round(rng.standard_normal((200, 16)) * 2.0 ** rng.integers(-6, 6, (200, 1)) * 64) / 64
    y, place = ref.rounded(x)
    for row, got, s in zip(x, y, place):
        a = np.abs(row).max()
        d = np.abs(ref.SCALES - a / 6)
        assert d[s] == d.min()
        step = ref.SCALES[s]
        if step == 0:
            assert (got == 0).all()
            continue
        grid = np.concatenate([-ref.CODES[::-1], ref.CODES]) * step
        best = np.abs(row[:, None] - grid).min(1)
        assert np.allclose(np.abs(row - got), best, rtol=1e-12, atol=0)


def test_reference_fork_keeps_histories():
    table = np.array([[3, 5, -1], [3, 7, 8], [-1, -1, -1]], np.int32)
    new, ln, used, copies = ref.fork(table, np.array([20, 40, 0]), np.array([0, 0, 1, -1, 2]),
                                     np.array([20, 40, 41, 0, 1]), 16, 12)
    assert ln.tolist() == [20, 20, 40, 0, 0]
    assert new.tolist() == [[3, 5, -1], [3, 0, 1], [3, 7, 8], [-1, -1, -1], [2, -1, -1]]
    assert copies == [(5, 0)] and used == 7  # 0, 1, 2, 3, 5, 7 and 8
