"""CPU checks: the calls on the 4-bit cache and on beams refuse outputs that overlap
any of their inputs (every call below fails validation before any CUDA call)."""
import pytest

import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build
from test_tree_forward_abi import FAKE, INVALID, WORKSPACE, caller

FAR = [FAKE + (i << 30) for i in range(1, 11)]


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return sv.load_library()


def test_commit(lib):
    call = caller(lib.spec_kv4_commit_path, pages=FAR[0], layers=2, n_pages=9, page=16, Hkv=2, D=64, table=FAR[1], W=3,
                  nk=FAR[2], nv=FAR[3], base=FAR[4], acc=FAR[5], path=FAR[6], md=4, exps=FAR[9], B=2, N=8, new=FAR[7],
                  ws=FAR[8], wsb=256, stream=None)
    nodes = 2 * 2 * 8 * 2 * 64 * 2
    for over in (FAR[9], FAR[9] + 12, FAR[2], FAR[2] + nodes - 4, FAR[3] - 4, FAR[3] + nodes - 4):
        assert call(new=over) == INVALID, over


@pytest.mark.parametrize("N", [1, 60])
def test_attention(lib, N):
    n = sv.spec_tree_attention_kv4_workspace_bytes(2, N, 8, 2, 64)
    names = dict(q=FAR[0], pages=FAR[1], table=FAR[2], nk=FAR[3], nv=FAR[4], mask=FAR[5], base=FAR[6], exps=FAR[7])
    call = caller(lib.spec_tree_attention_kv4, q=FAR[0], pages=FAR[1], n_pages=9, page=16, table=FAR[2], W=3, nk=FAR[3],
                  nv=FAR[4], mask=FAR[5], base=FAR[6], exps=FAR[7], B=2, N=N, Hq=8, Hkv=2, D=64, scale=0.1, out=FAR[8],
                  lse=FAR[8] + (1 << 29), ws=FAR[9], wsb=n, stream=None)
    last = dict(q=2 * N * 8 * 64 * 2, pages=9 * 2 * 9 * 16 * 64 // 8, table=24, nk=2 * N * 2 * 64 * 2,
                nv=2 * N * 2 * 64 * 2, mask=2 * N * ((N + 31) // 32) * 4, base=8, exps=8)
    for name, at in names.items():
        assert call(lse=at) == INVALID and call(lse=at + last[name] - 4) == INVALID, name
        assert call(lse=at - 2 * N * 8 * 4 + 4) == INVALID, name
        assert call(out=at) == INVALID and call(out=at + (last[name] - 1) // 16 * 16) == INVALID, name


def test_beams(lib):
    n = sv.spec_beam_select_workspace_bytes(2, 4, 1000, 4, 1)
    call = caller(lib.spec_beam_select, z=FAR[0], dtype=1, s=FAR[1], fin=FAR[2], eos=2, T=1.0, B=2, K=4, V=1000, M=4,
                  os=FAR[3], op=FAR[4], ot=FAR[5], of=FAR[6], ws=FAR[7], wsb=n, stream=None)
    for name in ("os", "op", "ot", "of"):
        for over in (FAR[0], FAR[0] - 28, FAR[0] + 2 * 4 * 1000 * 2 - 4):
            assert call(**{name: over}) == INVALID, (name, over)
    assert call(ws=None) == WORKSPACE
