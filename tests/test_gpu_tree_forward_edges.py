"""Edges of the tree's verification forward on the GPU: workspaces of exactly the
size asked for, values that are not finite, draws among very unlikely tokens,
waits that run out, and calls that the documentation allows at its limits."""
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
