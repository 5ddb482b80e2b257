"""Beam selection on the GPU where logits tie: zeros of both signs."""
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


def select(z, M, dtype):
    z = torch.from_numpy(z.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    r = sv.beam_select(z, torch.zeros(z.shape[:2], device="cuda"), M)
    return r["parents"].cpu().numpy(), r["tokens"].cpu().numpy()


# 1003: rows that are no whole number of vectors; 400000: more runs than a warp
# has shared memory for
@pytest.mark.parametrize("V", [1024, 1003, 20000, 400000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_of_both_signs_tie(V, dtype):
    """-0 and +0 are the same logit, so that the lowest tokens win: with a -0 in
    front of its lane's, other lanes' and other runs' +0, with any mixture of the
    signs, and with zeros among smaller logits."""
    rng = np.random.default_rng(V)
    rows = [np.zeros(V) for _ in range(6)]
    rows[0][0] = -0.0                                    # within a lane and across lanes
    rows[1][: min(V // 2, 700)] = -0.0                   # whole runs of -0 in front
    rows[2][:] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    rows[3][:] = -0.0
    rows[3][V - 1] = 0.0                                 # the one +0 comes last
    rows[4][:] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    rows[4][: V // 3] = -1.0
    rows[5][:] = -2.0
    few = np.sort(rng.choice(V, 20, replace=False))      # as many as fit a warp's lanes
    rows[5][few] = np.where(rng.random(20) < 0.5, 0.0, -0.0)
    first = [np.arange(16)] * 4 + [V // 3 + np.arange(16), few[:16]]
    z = np.stack(rows)[:, None, :]
    for M in (1, 7, 16):
        parents, tokens = select(z, M, dtype)
        for b in range(6):
            assert tokens[b].tolist() == first[b][:M].tolist(), (b, M)
            assert (parents[b] == b).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beams_whose_zeros_differ_in_sign_tie(dtype):
    """Rows that differ in the signs of zeros have the same totals: the lower beam
    comes first, with its lowest tokens."""
    V = 2000
    z = np.zeros((1, 3, V))
    z[0, 0] = -0.0
    z[0, 1, ::2] = -0.0
    parents, tokens = select(z, 16, dtype)
    assert (parents == 0).all() and tokens[0].tolist() == list(range(16))
