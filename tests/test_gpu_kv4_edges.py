"""The 4-bit cache in pages on the GPU at the ends of its arguments' ranges."""
import numpy as np
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


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_commit_of_lengths_at_the_ends_of_their_type():
    """Lengths that no sequence has: left untouched, new_len = max(base_len - 1, 0)."""
    base = np.array([-2**31, -2**31 + 1, -1, 0, 2**31 - 1, 5], np.int32)
    B, N, page, D = len(base), 3, 16, 64
    pages = sv.alloc_kv4_pages(1, B, 1, page, D)
    kv = torch.ones(1, B, N, 1, D, dtype=torch.bfloat16, device="cuda")
    table = cuda(np.arange(B, dtype=np.int32)[:, None])
    ws = sv.alloc_workspace(sv.SPEC_MODE_KV4, B, N, 1, sv.SPEC_DTYPE_BF16)
    n = sv.kv4_commit_path(pages, table, kv, kv, cuda(base), workspace=ws)
    assert n.tolist() == [0, 0, 0, 0, 2**31 - 2, 7]
    assert sv.spec_verify_read_flags(ws) == sv.SPEC_FLAG_BAD_PATH | sv.SPEC_FLAG_BAD_PAGE
    assert (pages[0, :5] == 0).all() and (pages[0, 5] != 0).any()
