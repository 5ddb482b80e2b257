"""Beam selection on the GPU where logits tie (zeros of both signs), and where they lie
far from zero or from one another."""
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


def check(z, scores, M, dtype, T=1.0, finished=None, eos=-1):
    """Every place against totals in 64 bits, whatever lies close together: within a
    beam exactly its largest logits, lower tokens first; a place's score is its
    candidate's total to 2^-18 + 2^-24 of what its logit lies below the row's largest
    (over T) and half a step of float32; no place and no candidate left out has a
    total that is smaller (larger) than a later place's (the last one's) by more."""
    z = torch.from_numpy(z.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    B, K, V = z.shape
    got = {n: x.cpu().numpy() for n, x in sv.beam_select(
        z, cuda(scores.astype(np.float32)), M, None if finished is None else cuda(finished.astype(np.int32)), eos, T).items()}
    z, T = z.double().cpu().numpy(), float(np.float32(T))
    scores = scores.astype(np.float32).astype(np.float64)
    for b in range(B):
        rows = []  # of each beam: its candidates in order, as (total, token, bound)
        for k in range(K):
            if not scores[b, k] > -np.inf:
                rows.append([])
            elif finished is not None and finished[b, k]:
                rows.append([(scores[b, k], eos, 0.0)])
            else:
                top = z[b, k].max()
                if top == -np.inf:
                    rows.append([])
                    continue
                y = (z[b, k] - top) / T
                total = scores[b, k] + (y - np.log(np.exp(y).sum()))
                order = np.lexsort((np.arange(V), -z[b, k]))[: M + 1]
                rows.append([(total[i], int(i), 2.0 ** -18 + 2.0 ** -24 * -y[i]) for i in order if z[b, k, i] > -np.inf])
        n = min(M, sum(len(r) for r in rows))
        assert (got["parents"][b, n:] == -1).all() and (got["tokens"][b, n:] == -1).all()
        assert (got["scores"][b, n:] == -np.inf).all() and (got["finished"][b, n:] == 1).all()
        at, places = [0] * K, []
        for i in range(n):
            k = int(got["parents"][b, i]) - b * K
            assert 0 <= k < K and at[k] < len(rows[k]), (b, i, k)
            total, token, bound = rows[k][at[k]]
            at[k] += 1
            assert got["tokens"][b, i] == token, (b, i, k)
            with np.errstate(over="ignore"):
                want = np.float32(total)
            off = abs(float(got["scores"][b, i]) - total)
            assert got["scores"][b, i] == want or off <= bound + 2.0 ** -24 * abs(total), (b, i, off, bound)
            done = finished is not None and finished[b, k]
            assert got["finished"][b, i] == int(bool(done) or token == eos)
            places.append((total, bound))
        left = [r[a] for r, a in zip(rows, at) if a < len(r)]
        for (x, bx), (y, by) in zip(places, places[1:]):
            assert x + bx >= y - by
        for y, _, by in left:
            assert places[-1][0] + places[-1][1] >= y - by, b
    return got


@pytest.mark.parametrize("V", [1000, 1003, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_far_from_zero(V, dtype):
    """Rows masked with the type's lowest value, in all places or in most, and rows of
    huge logits of either sign: totals are relative to the row's largest logit."""
    rng = np.random.default_rng(V)
    low = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min
    z = rng.standard_normal((9, 3, V)) * 2
    z[0, 1] = low                                  # a beam whose every token is masked
    z[1] = low                                     # all beams
    z[2, :, 5:] = low                              # five tokens left
    z[3, 0] = -1e30
    z[3, 1, : V // 2] = -1e38                      # chunks of other maxima, all far below
    z[3, 1, V // 2:] = -1e31
    z[4, 0] = 1e30
    z[4, 1, ::3] = 1e35
    z[5, 2] = np.where(rng.random(V) < 0.01, 3e38, -3e38)
    z[6] *= 1e9
    z[7] = z[7] * 1e8 - 3e9
    z[8, 0, : V - 1] = -np.inf                     # one token a beam, huge
    z[8, 0, V - 1] = -1e33
    scores = -rng.random((9, 3)) * 10
    for M in (1, 4, 16):
        check(z, scores, M, dtype)
        check(z, scores, M, dtype, T=0.3)


@pytest.mark.parametrize("T", [1e-3, 1e-6, 1e-9, 1e-20, 1e-38, 1e6, 1e30])
def test_temperatures_far_from_one(T):
    rng = np.random.default_rng(4)
    z = rng.standard_normal((3, 4, 5000)) * 3
    z[1, 2] = 0.0
    z[2, 1, 100:200] = z[2, 1].max() + 1
    for dtype in ("bf16", "f32"):
        check(z, -rng.random((3, 4)) * 5, 8, dtype, T=T)
        check(z * min(T * 1e9, 1e30), -rng.random((3, 4)) * 5, 8, dtype, T=T)  # (about 2^30 of it)
        check(z * min(T, 1e30), -rng.random((3, 4)) * 5, 8, dtype, T=T)


@pytest.mark.parametrize("T", [1.0, 0.9, 0.7, 1.3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_totals_of_candidates_far_below_the_largest(T, dtype):
    """Rows of few tokens with 10 to 1000 between them, so that the places go far
    down; and peaked, flat and long rows."""
    rng = np.random.default_rng(int(10 * T))
    z = np.full((8, 3, 3000), -np.inf)
    for b in range(4):
        n = 6
        z[b, :, rng.choice(3000, n, replace=False)] = rng.random((n, 3)) * 10.0 ** b
    z[4] = rng.standard_normal((3, 3000)) * 30
    z[5] = rng.standard_normal((3, 3000)) * 0.01
    z[6] = np.log(rng.random((3, 3000)))
    z[7, :, :16] = -np.arange(16) * 100.0 * T + np.array([[0.0], [1.0], [500.0]])
    for M in (3, 16):
        check(z, -rng.random((8, 3)) * 3, M, dtype, T=T)
    check(rng.standard_normal((2, 2, 151936)) * 3, -rng.random((2, 2)), 16, dtype, T=T)


@pytest.mark.parametrize("V", [500, 4099, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_place_holds_the_candidate_it_names(V, dtype):
    """Many close totals: parents and tokens are checked against their own totals,
    with finished beams, beams without a score, and an end token."""
    rng = np.random.default_rng(V)
    z = rng.standard_normal((4, 8, V))
    scores = -rng.random((4, 8)) * 0.5
    scores[1, 3] = -np.inf
    finished = rng.random((4, 8)) < 0.25
    for T in (1.0, 0.6):
        check(z, scores, 16, dtype, T=T, finished=finished, eos=min(7, V - 1))
