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


def host(t):
    return t.detach().double().cpu().numpy()


def in_half(x, e):
    """x as fp16 in units of 2^e, where its 8 bits do not fit: multiples of 2^-24."""
    y = x * 2.0 ** -e
    return np.clip(np.where(np.abs(y) < 2.0 ** -14, np.rint(y * 2.0 ** 24) * 2.0 ** -24, y), -65504, 65504) * 2.0 ** e


@pytest.mark.parametrize("Hq,D", [(2, 64), (2, 128), (64, 64), (64, 128)])  # few rows, and tiles
@pytest.mark.parametrize("e", [0, -20, 31])
def test_a_node_alone_has_the_documented_precision(Hq, D, e):
    """One node that sees itself alone: its weight is 1 (2^7 in fp16, both exact), so
    that the output is the value as the products take it: exact from 2^-17 2^e on,
    multiples of 2^-24 2^e below, at most 65504 2^e (rounded to bf16: 2^16)."""
    B, Hkv, page = 60, 2, 16
    rng = np.random.default_rng(D + e)
    mag = np.exp2(np.arange(B) - 35.0 + e)[:, None, None, None]  # 2^-35 .. 2^24 of 2^e
    nv = torch.from_numpy((rng.choice([-1, 1], (B, 1, Hkv, D)) * rng.integers(128, 256, (B, 1, Hkv, D)) / 128.0 * mag)
                          .astype(np.float32)).bfloat16().cuda()
    q, nk = (torch.randn(B, 1, h, D, device="cuda").bfloat16() for h in (Hq, Hkv))
    exps = cuda(np.array([0, e], np.int32))
    pages, table = sv.alloc_kv4_pages(1, 1, Hkv, page, D), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    out, _ = sv.tree_attention_kv4(q, pages[0], table, nk, nv, None, torch.ones(B, dtype=torch.int32, device="cuda"),
                                   kv_exp=exps)
    want = torch.from_numpy(in_half(host(nv), e)).repeat_interleave(Hq // Hkv, dim=2)
    want = want.to(torch.float32).bfloat16().double()  # (exact but for 65504)
    assert np.array_equal(host(out), want.numpy())


@pytest.mark.parametrize("N,D", [(1, 64), (5, 128), (40, 64), (60, 128)])
@pytest.mark.parametrize("mag", [-13, -18, -22, -26])
@pytest.mark.parametrize("exps", [(0, 0), (-9, 12)])
def test_attention_of_small_nodes(N, D, mag, exps):
    """Nodes far below the layer's exponents, alone and behind committed positions.
    To what the other attention tests allow: keys are off by up to 2^-25 2^e in each
    channel, a score by that times scale sum |q|, values by up to 2^-25 2^e."""
    import kv4_reference as ref
    from test_gpu_kv4 import Case
    c = Case(3, N, 8, 2, D, 32, [1, 40, 150], False, exps=exps)
    c.nk = (c.nk.float() * 2.0 ** (exps[0] + mag)).bfloat16()
    c.nv = (c.nv.float() * 2.0 ** (exps[1] + mag)).bfloat16()
    c.scale = 2.0 ** (-exps[0] - mag) / D  # scores of the nodes of the order of 1
    c.pages = c.pages.copy()
    blocks = c.pages.reshape(len(c.pages), 2, 2, 2, 9 * D)
    blocks[:, :, :, 0, 8 * D:] = 0         # (committed keys 0: their scores would drown those)
    out, lse = (host(x) for x in c.run())
    for b in range(3):
        n = int(c.base[b]) - 1
        k, v = ref.unpack(c.pages, c.table[b], n, 32, D, exps)
        k, v = np.concatenate([k, host(c.nk[b])]), np.concatenate([v, host(c.nv[b])])
        sees = np.concatenate([np.ones((N, n), bool), c.anc[b]], 1)
        q = host(c.q[b])
        o, l, mass, amp = ref.attention(q, k, v, sees, c.scale)
        ds = D * 2.0 ** -23 * amp + 4e-5 + c.scale * np.abs(q).sum(2) * 2.0 ** (exps[0] - 25)
        assert (np.abs(lse[b] - l) <= ds + 2.0 ** -22 * np.abs(l)).all()
        small = 2.0 ** -32 * np.repeat(np.abs(v).sum(0), 4, axis=0) + 2.0 ** (exps[1] - 25)
        tol = 2.0 ** -8 * np.abs(o) + (3 * 2.0 ** -11 + 2 * ds[..., None]) * mass + small
        assert (np.abs(out[b] - o) <= tol).all()
