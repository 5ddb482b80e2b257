"""CPU checks of the tree's verification forward: workspace sizes and the host's
refusals (every call below fails validation or is the B = 0 no-op, before any
CUDA call), and the Python wrappers' refusals that need no GPU."""
import pytest

import speculative_decoding_verification_56_gb300 as sv
from speculative_decoding_verification_56_gb300 import build

FAKE = 0x10000          # 64 KiB-aligned fake device address, never dereferenced
OK, INVALID, ALIGN, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return sv.load_library()


def caller(fn, **defaults):
    def call(**over):
        assert not set(over) - set(defaults)
        return fn(*{**defaults, **over}.values())
    return call


def test_workspace_sizes(lib):
    ws = sv.spec_verify_workspace_bytes
    assert ws(sv.SPEC_MODE_TREE_SAMPLE, 16, 60, 128256, sv.SPEC_DTYPE_BF16) == 256
    assert ws(sv.SPEC_MODE_TREE_QKV, 16, 60, 1, sv.SPEC_DTYPE_BF16) == 256
    assert ws(sv.SPEC_MODE_TREE_SAMPLE, 16, 0, 10, 0) == 0
    at = sv.spec_tree_attention_workspace_bytes
    a, b = at(16, 60, 32, 8, 128), at(32, 60, 32, 8, 128)
    assert 0 < a < b and a % 256 == 0
    assert at(16, 60, 32, 8, 128, 8192) > a          # partials of the shared prefix
    assert at(64, 1, 32, 8, 128) < 16 << 20           # decoding keeps few rows a slot
    for bad in ((-1, 60, 32, 8, 128, 0), (1, 0, 32, 8, 128, 0), (1, 4097, 32, 8, 128, 0),
                (1, 1, 30, 8, 128, 0), (1, 1, 8, 0, 128, 0), (1, 1, 129, 1, 128, 0),
                (1, 1, 32, 8, 96, 0), (1, 1, 32, 8, 128, -1), (1 << 24, 4096, 32, 8, 128, 0)):
        assert at(*bad) == 0, bad


def test_tree_sample_validation(lib):
    call = caller(lib.spec_verify_tree_sample, z=FAKE, dtype=1, tok=FAKE, par=FAKE, u=FAKE, T=1.0, B=2, N=8,
                  V=100, md=4, n=FAKE, path=FAKE, out=FAKE, probs=FAKE, ws=FAKE, wsb=256, stream=None)
    for over in (dict(dtype=2), dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")),
                 dict(B=-1), dict(N=0), dict(N=65537), dict(V=0), dict(V=(1 << 26) + 1), dict(md=-1),
                 dict(md=1025), dict(B=1 << 28), dict(z=None), dict(tok=None), dict(par=None),
                 dict(u=None), dict(n=None), dict(path=None), dict(out=None), dict(probs=None)):
        assert call(**over) == INVALID, over
    for over in (dict(z=FAKE + 1), dict(dtype=0, z=FAKE + 2), dict(tok=FAKE + 2), dict(u=FAKE + 1),
                 dict(probs=FAKE + 2), dict(ws=FAKE + 16)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE
    assert call(B=0, z=None, tok=None, ws=None, wsb=0) == OK


def test_tree_qkv_validation(lib):
    call = caller(lib.spec_tree_qkv_rope, qkv=FAKE, qn=FAKE, kn=None, eps=1e-6, freq=FAKE, rot=64, inter=0,
                  off=0, base=FAKE, depth=None, B=2, N=8, Hq=8, Hkv=2, D=64, L=100, stride=100 * 2 * 64 * 2,
                  q=FAKE, k=FAKE, v=FAKE, ws=FAKE, wsb=256, stream=None)
    for over in (dict(B=-1), dict(N=0), dict(N=65537), dict(Hq=0), dict(Hkv=0), dict(D=96), dict(L=0),
                 dict(rot=-2), dict(rot=66), dict(rot=7), dict(off=-1), dict(off=1 << 31), dict(eps=-1e-6),
                 dict(eps=float("nan")), dict(stride=100 * 2 * 64 * 2 - 16), dict(B=1 << 20, N=65536),
                 dict(qkv=None), dict(base=None), dict(q=None), dict(k=None), dict(v=None), dict(freq=None)):
        assert call(**over) == INVALID, over
    for over in (dict(qkv=FAKE + 8), dict(q=FAKE + 8), dict(k=FAKE + 4), dict(v=FAKE + 8), dict(qn=FAKE + 2),
                 dict(kn=FAKE + 8), dict(stride=100 * 2 * 64 * 2 + 8), dict(base=FAKE + 1),
                 dict(depth=FAKE + 2), dict(ws=FAKE + 16)):
        assert call(**over) == ALIGN, over
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE
    assert call(B=0, qkv=None, ws=None) == OK
    assert call(rot=0, freq=None, wsb=16) == WORKSPACE   # no frequencies are needed then


def test_tree_attention_validation(lib):
    call = caller(lib.spec_tree_attention, q=FAKE, k=FAKE, v=FAKE, stride=100 * 2 * 64 * 2, L=100, pk=None,
                  pv=None, P=0, mask=None, base=FAKE, B=2, N=8, Hq=8, Hkv=2, D=64, scale=0.125, out=FAKE,
                  lse=None, ws=FAKE, wsb=1 << 30, stream=None)
    for over in (dict(B=-1), dict(N=0), dict(N=4097), dict(Hq=7), dict(Hq=1), dict(Hkv=0), dict(D=32),
                 dict(Hq=258), dict(L=0), dict(L=2 ** 31 - 100), dict(P=-1), dict(scale=0.0),
                 dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                 dict(stride=100 * 2 * 64 * 2 - 16), dict(P=5), dict(P=5, pk=FAKE), dict(q=None),
                 dict(k=None), dict(v=None), dict(base=None), dict(out=None)):
        assert call(**over) == INVALID, over
    for over in (dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(out=FAKE + 8),
                 dict(stride=100 * 2 * 64 * 2 + 8), dict(P=5, pk=FAKE, pv=FAKE + 8), dict(mask=FAKE + 2),
                 dict(base=FAKE + 2), dict(lse=FAKE + 1), dict(ws=FAKE + 16)):
        assert call(**over) == ALIGN, over
    need = sv.spec_tree_attention_workspace_bytes(2, 8, 8, 2, 64)
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(B=0, q=None, ws=None, wsb=0) == OK


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros(1, 2, 8)
    i = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_verify_tree_sample(z, i, i, torch.zeros(1, 3), 1.0, 2, i, i, i, z, i)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q, kc, kc, None, i[0], 1.0, q, None, i)
    with pytest.raises(ValueError):
        sv.spec_tree_qkv_rope(q, None, None, 1e-6, z, i, None, q, kc, kc, i)


def test_tree_attention_scale_stays_finite(lib):
    call = caller(lib.spec_tree_attention, q=FAKE, k=FAKE, v=FAKE, stride=100 * 2 * 64 * 2, L=100, pk=None,
                  pv=None, P=0, mask=None, base=FAKE, B=2, N=8, Hq=8, Hkv=2, D=64, scale=0.125, out=FAKE,
                  lse=None, ws=FAKE, wsb=0, stream=None)
    assert call(scale=2.0 ** 127) == INVALID and call(scale=3e38) == INVALID
    assert call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    assert call(scale=1.5 * 2.0 ** 126) == WORKSPACE and call(scale=1e-45) == WORKSPACE


@pytest.mark.parametrize("B,N,Hq,Hkv,D,P", [
    (64, 1, 32, 8, 128, 0), (64, 1, 32, 8, 128, 1), (1024, 1, 32, 8, 128, 1), (256, 60, 32, 8, 128, 0),
    (256, 60, 32, 8, 128, 8192), (1, 5, 8, 8, 64, 0), (20, 1, 8, 8, 64, 0), (3, 200, 71, 1, 64, 129),
])
def test_attention_workspace_holds_what_the_join_reads(lib, B, N, Hq, Hkv, D, P):
    """Slots of an item's own rows: one part of every item behind a shared prefix
    and one more a CTA (of the larger kind); without a prefix two a CTA at most."""
    ctas, tok = 160, 128 // (Hq // Hkv)

    def items_and_rows(nodes):
        per = 2 * tok if nodes > tok else tok
        return -(-nodes // per), min(nodes, per) * (Hq // Hkv)

    mg, rows = items_and_rows(N)
    items = B * Hkv * mg
    held = (items + ctas if P else min(items + ctas, 2 * ctas)) * rows
    if P:
        mg, rows = items_and_rows(B * N)
        held += Hkv * mg * rows + ctas * (rows - min(N, 2 * tok if N > tok else tok) * (Hq // Hkv))
        items += Hkv * mg
    need = 256 + items * 8 + held * (4 * D + 8)     # flags, spans; row: D floats, reference and sum
    got = sv.spec_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, P)
    assert need <= got < need + 4 * 256             # parts start at multiples of 256


def test_device_getters_without_torch_internals():
    from types import SimpleNamespace as NS
    public = NS(_C=NS(), cuda=NS(current_device=lambda: 3, current_stream=lambda i: NS(cuda_stream=100 + i)))
    device, stream = sv._device_getters(public)
    assert device() == 3 and stream(2) == 102
    public._C = NS(_cuda_getDevice=lambda: 1, _cuda_getCurrentRawStream=lambda i: 200 + i)
    device, stream = sv._device_getters(public)
    assert device() == 1 and stream(2) == 202


def test_conveniences_refuse_caches_of_another_rank(lib):
    torch = pytest.importorskip("torch")
    bf16 = dict(dtype=torch.bfloat16)
    qkv, q = torch.zeros(1, 2, 8, 64, **bf16), torch.zeros(1, 2, 4, 64, **bf16)
    one = torch.ones(1, dtype=torch.int32)
    for cache in (torch.zeros(9, 64, **bf16), torch.zeros(1, 9, 64, **bf16), torch.zeros(1, 1, 9, 2, 64, **bf16)):
        with pytest.raises(ValueError, match="k_cache"):
            sv.tree_qkv_rope(qkv, None, None, 1e-6, None, one, None, cache, cache)
        with pytest.raises(ValueError, match="k_cache"):
            sv.tree_attention(q, cache, cache, None, one)
    four = torch.zeros(1, 9, 4, 64, **bf16)
    with pytest.raises(ValueError, match="no query head"):
        sv.tree_qkv_rope(qkv, None, None, 1e-6, None, one, None, four, four)


def test_attention_workspace_is_never_more_than_slots_of_one_size(lib):
    """items + CTAs slots that all hold the largest kind's rows."""
    for B in (1, 2, 17, 64, 1000):
        for N in (1, 5, 33, 60, 500):
            for Hq, Hkv in ((8, 8), (32, 8), (71, 1), (15, 3)):
                for P in (0, 1, 5000):
                    G, tok = Hq // Hkv, 128 // (Hq // Hkv)

                    def per(nodes):
                        return 2 * tok if nodes > tok else tok
                    items = B * Hkv * -(-N // per(N)) + (Hkv * -(-B * N // per(B * N)) if P else 0)
                    rows = min(tok, B * N if P else N) * G * (2 if max(N, B * N if P else 0) > tok else 1)
                    most = 256 + items * 8 + (items + 160) * rows * (4 * 128 + 8) + 4 * 256
                    assert sv.spec_tree_attention_workspace_bytes(B, N, Hq, Hkv, 128, P) <= most, (B, N, Hq, Hkv, P)
