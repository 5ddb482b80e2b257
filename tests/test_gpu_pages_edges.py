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


@pytest.mark.parametrize("B,B2,W,page,n_pages", [
    (1, 4, 5, 16, 40), (8, 8, 7, 32, 90), (5, 17, 6, 1, 20), (64, 64, 18, 64, 700), (64, 64, 18, 64, 1400),
    (3, 512, 4, 3, 600), (200, 300, 9, 128, 1100), (600, 600, 5, 16, 4000), (600, 600, 5, 16, 1500),
    (10, 12, 6, 16, 40000), (20, 9, 5000, 16, 60000), (4, 1500, 6, 16, 2000), (900, 2100, 3, 16, 2500),
])
def test_fork_flags_and_exclusive_pages(B, B2, W, page, n_pages):
    """The flag says that no page was left exactly where an entry is missing, and with
    pages left or not, every position to come stands in a page of its sequence alone."""
    import numpy as np
    from test_gpu_pages_beams import check_fork, tables
    rng = np.random.default_rng(B + B2 + W + n_pages)
    table, length = tables(rng, B, W, page, n_pages)
    parent = rng.integers(-1, B, B2).astype(np.int32)
    need = np.where(parent >= 0, np.minimum(length[parent] + rng.integers(0, 2 * page, B2), W * page), 0).astype(np.int32)
    flags, new, ln = check_fork(rng, table, length, parent, need, page, n_pages)
    want = -(-np.maximum(need, ln) // page)
    missing = (new < 0) & (np.arange(W) < want[:, None])
    assert flags == (sv.SPEC_FLAG_NO_PAGE if missing.any() else 0)
    assert (new[np.arange(W) >= want[:, None]] == -1).all() and (new < n_pages).all()
    holders = np.bincount(new[new >= 0], minlength=n_pages)
    to_come = (new >= 0) & ((np.arange(W) + 1) * page > ln[:, None])
    assert (holders[new[to_come]] == 1).all()
