"""Empty batches of the calls on the 4-bit cache, on pages and on beams."""
import pytest
import torch

import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()
    sv.load_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("N", [1, 60])
def test_no_sequences(N):
    pages = sv.alloc_kv4_pages(2, 5, 2, 16, 64)
    pages[:] = 7
    old = pages.clone()
    out, lse = sv.tree_attention_kv4(bf16(0, N, 8, 64), pages[0], i32(0, 3), bf16(0, N, 2, 64), bf16(0, N, 2, 64), None, i32(0))
    assert out.shape == (0, N, 8, 64) and lse.shape == (0, N, 8)
    q, k, v = sv.tree_qkv_rope_nodes(bf16(0, N, 12, 64), 2, None, None, 0.0, None, i32(0), None)
    assert q.shape == (0, N, 8, 64) and k.shape == v.shape == (0, N, 2, 64)
    assert sv.kv4_commit_path(pages, i32(0, 3), bf16(2, 0, N, 2, 64), bf16(2, 0, N, 2, 64), i32(0)).numel() == 0
    k, v = sv.kv4_read(pages, i32(0, 3), i32(0), 40, 64)
    assert k.shape == v.shape == (2, 0, 40, 2, 64)
    r = sv.beam_select(torch.zeros(0, 3, 100, device="cuda"), torch.zeros(0, 3, device="cuda"), 4)
    assert r["scores"].shape == (0, 4)
    table, length, used = sv.kv_pages_fork(pages, i32(0, 3), i32(0), i32(0), None, 16)
    assert table.shape == (0, 3) and length.numel() == 0 and int(used) == 0
    table, used = sv.kv_pages_compact(pages, i32(0, 3))
    assert table.shape == (0, 3) and int(used) == 0
    torch.cuda.synchronize()
    assert torch.equal(pages, old)


def test_forks_from_no_sequences():
    """Rows that are all empty need no old table; one that names a parent is flagged."""
    pages = torch.zeros(1, 6, 16, dtype=torch.uint8, device="cuda")
    ws = sv.alloc_kv_pages_workspace(pages, 2)
    table, length, used = sv.kv_pages_fork(pages, i32(0, 3), i32(0), i32(2) - 1, i32(2) + 40, 16, ws)
    assert (table == -1).all() and length.tolist() == [0, 0] and int(used) == 0
    assert sv.spec_verify_read_flags(ws) == 0
    table, _, used = sv.kv_pages_fork(pages, i32(0, 3), i32(0), i32(2), i32(2) + 40, 16, ws)
    assert (table == -1).all() and int(used) == 0 and sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PARENT
