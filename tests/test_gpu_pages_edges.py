"""Forks of pages on the GPU that ask for more pages than 32 bits count."""
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


def test_fork_that_wants_more_than_2_31_pages():
    """2049 sequences of 2^20 pages each, of a pool of 40: the first gets what there
    is, all others -1 (a table of 8.6 GB)."""
    rows, W, n_pages = 2049, sv.SPEC_KV_MAX_TABLE, 40
    assert rows * W > 1 << 31
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = torch.arange(n_pages * 4, **i32).view(1, n_pages, 4)
    old = pages.clone()
    table = torch.full((1, W), -1, **i32)
    table[0, 0] = 7
    parent = torch.zeros(rows, **i32)
    ws = sv.alloc_kv_pages_workspace(pages, rows)
    # one position in a page of one: page 7 is shared by all
    new, length, used = sv.kv_pages_fork(pages, table, torch.ones(1, **i32), parent, torch.full((rows,), W, **i32), 1, ws)
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_NO_PAGE
    assert new[0, : n_pages + 1].tolist() == [7] + [i for i in range(n_pages) if i != 7] + [-1]
    assert (new[0, n_pages:] == -1).all() and (new[1:, 0] == 7).all()
    for b in range(1, rows, 256):  # (a few rows at a time: comparisons take room)
        assert (new[b: b + 256, 1:] == -1).all()
    assert (length == 1).all() and int(used) == n_pages and torch.equal(pages, old)
