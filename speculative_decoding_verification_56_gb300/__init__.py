"""GB300-native batched draft-token verification for speculative decoding.

Thin ctypes binding over ``libspecverify.so`` (C ABI in ``include/spec_verify.h``).
Every step of verification runs in the library's CUDA kernels; this module only
marshals torch CUDA tensors (device memory, streams) into pointers and sizes.
There is no CPU fallback: without the compiled library every call raises.

Entry points (same names as the C ABI):

* :func:`spec_verify_sample`      -- rejection-sampling verification of chains
* :func:`spec_verify_greedy`      -- greedy verification of chains
* :func:`spec_verify_tree_greedy` -- greedy verification of draft trees
* :func:`spec_tree_attention_mask` -- ancestor bitmask + depth of draft trees
* :func:`spec_kv_commit_path`     -- move the accepted path's KV entries into place
* :func:`spec_lm_head_verify_greedy` -- LM head (tcgen05 GEMM) fused with greedy verification
* :func:`spec_lm_head_verify_sample` -- LM head (tcgen05 GEMM) fused with sampling verification
* :func:`spec_tree_grow`          -- EAGLE-2 dynamic draft-tree growth
* :func:`spec_tree_qkv_rope`      -- head norms, rotation and cache write of the tree's nodes
* :func:`spec_tree_attention`     -- attention of the tree's nodes over the cache and a shared prefix
* :func:`spec_verify_tree_sample` -- sampling verification of draft trees
* :func:`spec_verify_workspace_bytes`, :func:`spec_tree_attention_workspace_bytes`,
  :func:`spec_verify_read_flags`,
  :func:`spec_verify_launch_count`, :func:`spec_status_string`

Convenience wrappers that also allocate outputs and a workspace with torch:
:func:`verify_sample`, :func:`verify_greedy`, :func:`verify_tree_greedy`,
:func:`tree_attention_mask`, :func:`lm_head_verify_greedy`,
:func:`lm_head_verify_sample`, :func:`tree_grow`, :func:`tree_qkv_rope`,
:func:`tree_attention`, :func:`verify_tree_sample`.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_ALIGNMENT = 2
SPEC_ERR_WORKSPACE = 3
SPEC_ERR_CUDA = 4
SPEC_ERR_TOO_LARGE = 5
SPEC_NOALLOC_SCRATCH_BYTES = 4 << 20
SPEC_DTYPE_F32 = 0
SPEC_DTYPE_BF16 = 1
SPEC_MODE_SAMPLE = 0
SPEC_MODE_GREEDY = 1
SPEC_MODE_TREE_GREEDY = 2
SPEC_MODE_TREE_MASK = 3
SPEC_MODE_KV_COMMIT = 4
SPEC_MODE_LM_HEAD_GREEDY = 5
SPEC_MODE_TREE_GROW = 6
SPEC_MODE_LM_HEAD_SAMPLE = 7
SPEC_MODE_TREE_SAMPLE = 8
SPEC_MODE_TREE_QKV = 10
SPEC_ATTN_MAX_NODES = 4096
SPEC_LM_MAX_D = 8192
SPEC_FLAG_TOKEN_RANGE = 1
SPEC_FLAG_BAD_PARENT = 2
SPEC_FLAG_DEPTH = 4
SPEC_FLAG_RESIDUAL_FALLBACK = 8
SPEC_FLAG_TIMEOUT = 16
SPEC_FLAG_BAD_PATH = 32
SPEC_FLAG_EMPTY_ROW = 64

_lock = threading.Lock()
_lib = None
_torch_module = None
_current_device = _raw_stream = None


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {spec_status_string(status)} (status {status})")


def load_library(path: str = LIB_PATH):
    """Load the compiled C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with "
                "`python -m speculative_decoding_verification_56_gb300.build`")
        lib = ctypes.CDLL(path)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.spec_verify_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.spec_verify_workspace_bytes.restype = Z
        lib.spec_verify_sample.argtypes = [P, P, I, P, P, P, F, I, I, I, P, P, P, P, P, P, Z, P]
        lib.spec_verify_sample.restype = I
        lib.spec_verify_greedy.argtypes = [P, I, P, I, I, I, P, P, P, Z, P]
        lib.spec_verify_greedy.restype = I
        lib.spec_verify_tree_greedy.argtypes = [P, I, P, P, I, I, I, I, P, P, P, P, Z, P]
        lib.spec_verify_tree_greedy.restype = I
        lib.spec_verify_greedy_noalloc.argtypes = [P, I, P, I, I, I, P, P, P]
        lib.spec_verify_greedy_noalloc.restype = I
        lib.spec_verify_selftest_exp2.argtypes = [P, P, P, I, P]
        lib.spec_verify_selftest_exp2.restype = I
        lib.spec_tree_attention_mask.argtypes = [P, I, I, P, P, P, Z, P]
        lib.spec_tree_attention_mask.restype = I
        LL = ctypes.c_longlong
        lib.spec_kv_commit_path.argtypes = [P, I, I, LL, LL, I, I, I, P, P, P, I, P, P, Z, P]
        lib.spec_kv_commit_path.restype = I
        lib.spec_lm_head_verify_greedy.argtypes = [P, P, P, I, I, I, I, P, P, P, Z, P]
        lib.spec_lm_head_verify_greedy.restype = I
        lib.spec_lm_head_verify_sample.argtypes = [P, P, P, P, P, P, F, I, I, I, I, P, P, P, P, P,
                                                   P, Z, P]
        lib.spec_lm_head_verify_sample.restype = I
        lib.spec_tree_grow.argtypes = [P, I, F, I, I, I, I, I, P, P, P, P, P, Z, P]
        lib.spec_tree_grow.restype = I
        lib.spec_verify_tree_sample.argtypes = [P, I, P, P, P, F, I, I, I, I, P, P, P, P, P, Z, P]
        lib.spec_verify_tree_sample.restype = I
        lib.spec_tree_qkv_rope.argtypes = [P, P, P, F, P, I, I, LL, P, P, I, I, I, I, I, I, LL, P,
                                           P, P, P, Z, P]
        lib.spec_tree_qkv_rope.restype = I
        lib.spec_tree_attention_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.spec_tree_attention_workspace_bytes.restype = Z
        lib.spec_tree_attention.argtypes = [P, P, P, LL, I, P, P, I, P, P, I, I, I, I, I, F, P, P,
                                            P, Z, P]
        lib.spec_tree_attention.restype = I
        lib.spec_verify_read_flags.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), I, P]
        lib.spec_verify_read_flags.restype = I
        lib.spec_verify_launch_count.argtypes = []
        lib.spec_verify_launch_count.restype = ctypes.c_uint64
        lib.spec_verify_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        lib.spec_verify_set_wait_limit_ns.restype = None
        lib.spec_status_string.argtypes = [I]
        lib.spec_status_string.restype = ctypes.c_char_p
        lib.spec_verify_abi_version.argtypes = []
        lib.spec_verify_abi_version.restype = I
        _lib = lib
        return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _torch():
    global _torch_module, _current_device, _raw_stream
    if _torch_module is None:
        import torch
        _current_device, _raw_stream = _device_getters(torch)
        _torch_module = torch
    return _torch_module


def _device_getters(torch):
    """Functions that give the current device's index and a device's current
    stream as an integer: torch's internal ones (a small rotation's call takes
    10.6 us with them, 11.4 with the public device getter) or, where a torch
    does not have them, the public ones."""
    device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return device, stream or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return SPEC_DTYPE_BF16
    if t.dtype == torch.float32:
        return SPEC_DTYPE_F32
    raise TypeError(f"logits must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _dev(t, name, dtype=None, optional=False):
    """Pointer of a contiguous CUDA tensor (None -> NULL when optional)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _arg(t, name, dtype, shape, device):
    """Pointer of a contiguous CUDA tensor of the given type and shape on the
    call's device."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    raise ValueError(f"{name} must be contiguous")


def _call_device(t, name):
    """Index of the CUDA device that a call runs on: its tensors' device, which
    has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    _torch()
    if dev != _current_device():  # (CUDA is initialised: t is there)
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return dev


def _cache_args(k_cache, v_cache, Hkv, D, B, device):
    """Pointers, byte stride between sequences and positions of a layer's key
    and value cache [B, L, Hkv, D] (sequences may lie further apart)."""
    bf16 = _torch().bfloat16
    shape, stride = k_cache.shape, k_cache.stride()
    if (k_cache.dtype is bf16 and v_cache.dtype is bf16 and len(shape) == 4
            and shape == (B, shape[1], Hkv, D) and v_cache.shape == shape
            and k_cache.get_device() == device and v_cache.get_device() == device
            and stride == (stride[0], Hkv * D, D, 1) and v_cache.stride() == stride):
        L = shape[1]
        step = stride[0] if B > 1 else max(stride[0], L * Hkv * D)
        return k_cache.data_ptr(), v_cache.data_ptr(), 2 * step, L
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype is not bf16:
            raise TypeError(f"{name} must be {bf16}, got {t.dtype}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}")
        if t.dim() != 4 or t.shape != (B, t.shape[1], Hkv, D):
            raise ValueError(f"{name} must be [{B}, L, {Hkv}, {D}], got {list(t.shape)}")
    raise ValueError("k_cache and v_cache must have the same shape and strides, with the positions "
                     "of a sequence contiguous")


def _cache_heads(k_cache):
    """Key-value heads of a cache, for the conveniences, which size their
    allocations by it before the call checks its arguments."""
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [B, L, heads, D], got {list(k_cache.shape)}")
    return k_cache.shape[2]


def _workspace(t, device):
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return t.data_ptr(), t.nbytes


def _stream_of(stream, device):
    """_stream_ptr for a call on a known device (the current one)."""
    if stream is not None:
        return _stream_ptr(stream)
    _torch()
    return _raw_stream(device)


def _stream_ptr(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status, where):
    if status != SPEC_OK:
        raise SpecVerifyError(status, where)


# ---------------------------------------------------------------------------
# C-ABI entry points
# ---------------------------------------------------------------------------

def spec_status_string(status: int) -> str:
    try:
        return load_library().spec_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def spec_verify_workspace_bytes(mode: int, B: int, k_or_N: int, V: int, dtype: int) -> int:
    return int(load_library().spec_verify_workspace_bytes(mode, B, k_or_N, V, dtype))


def spec_verify_launch_count() -> int:
    return int(load_library().spec_verify_launch_count())


def spec_verify_abi_version() -> int:
    return int(load_library().spec_verify_abi_version())


def spec_verify_set_wait_limit_ns(limit_ns: int) -> None:
    """Limit of the verification kernels' waits on their bulk copies, and of the
    tree attention's waits between its roles, for calls enqueued afterwards (0
    restores the default 0.2 s); a diagnostic control for testing the timeout
    path."""
    load_library().spec_verify_set_wait_limit_ns(int(limit_ns))


def spec_verify_sample(target_logits, draft_logits, draft_tokens, u_accept, u_sample,
                       temperature, accepted_len, out_tokens, p_out, q_out, resid_mass,
                       workspace, stream=None):
    """Rejection-sampling verification (C ABI ``spec_verify_sample``).

    target_logits [B, k+1, V] and draft_logits [B, k, V] (bf16 or fp32);
    draft_tokens int32 [B, k]; u_accept float32 [B, k]; u_sample float32 [B].
    Outputs (preallocated CUDA tensors): accepted_len int32 [B], out_tokens
    int32 [B, k+1], p_out/q_out float32 [B, k], resid_mass float32 [B].
    workspace: uint8 CUDA tensor of at least spec_verify_workspace_bytes() bytes.
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dt = _dtype_code(target_logits)
    if k > 0 and (draft_logits is None or draft_logits.dtype != target_logits.dtype
                  or tuple(draft_logits.shape) != (B, k, V)):
        raise ValueError("draft_logits must be [B, k, V] with the target's dtype")
    st = load_library().spec_verify_sample(
        _dev(target_logits, "target_logits"),
        _dev(draft_logits, "draft_logits", optional=k == 0), dt,
        _dev(draft_tokens, "draft_tokens", torch.int32, optional=k == 0),
        _dev(u_accept, "u_accept", torch.float32, optional=k == 0),
        _dev(u_sample, "u_sample", torch.float32), float(temperature), B, k, V,
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32),
        _dev(p_out, "p_out", torch.float32, optional=k == 0),
        _dev(q_out, "q_out", torch.float32, optional=k == 0),
        _dev(resid_mass, "resid_mass", torch.float32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_verify_sample")


def spec_verify_greedy(target_logits, draft_tokens, accepted_len, out_tokens, workspace,
                       stream=None):
    """Greedy verification (C ABI ``spec_verify_greedy``)."""
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    st = load_library().spec_verify_greedy(
        _dev(target_logits, "target_logits"), _dtype_code(target_logits),
        _dev(draft_tokens, "draft_tokens", torch.int32, optional=k == 0), B, k, V,
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_verify_greedy")


def spec_verify_greedy_noalloc(target_logits, draft_tokens, accepted_len, out_tokens,
                               stream=None):
    """Greedy verification on the library's fixed device scratch (C ABI
    ``spec_verify_greedy_noalloc``): for callers that cannot allocate device
    memory when they verify.  Calls sharing the scratch must not overlap."""
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    st = load_library().spec_verify_greedy_noalloc(
        _dev(target_logits, "target_logits"), _dtype_code(target_logits),
        _dev(draft_tokens, "draft_tokens", torch.int32, optional=k == 0), B, k, V,
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32), _stream_ptr(stream))
    _check(st, "spec_verify_greedy_noalloc")


def spec_verify_tree_greedy(target_logits, node_tokens, parents, max_depth, accepted_len,
                            path_nodes, out_tokens, workspace, stream=None):
    """Draft-tree greedy verification (C ABI ``spec_verify_tree_greedy``)."""
    torch = _torch()
    B, N, V = target_logits.shape
    st = load_library().spec_verify_tree_greedy(
        _dev(target_logits, "target_logits"), _dtype_code(target_logits),
        _dev(node_tokens, "node_tokens", torch.int32), _dev(parents, "parents", torch.int32),
        B, N, V, int(max_depth),
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(path_nodes, "path_nodes", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_verify_tree_greedy")


def spec_tree_attention_mask(parents, mask, depth, workspace, stream=None):
    """Tree attention mask (C ABI ``spec_tree_attention_mask``): ``mask``
    int32/uint32-sized [B, N, ceil(N/32)] words, ``depth`` int32 [B, N] or
    None."""
    torch = _torch()
    B, N = parents.shape
    st = load_library().spec_tree_attention_mask(
        _dev(parents, "parents", torch.int32), B, N, _dev(mask, "mask"),
        _dev(depth, "depth", torch.int32, optional=True),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_tree_attention_mask")


def spec_kv_commit_path(cache, base_len, accepted_len, path_nodes, N, new_len, workspace,
                        stream=None):
    """KV commit of the accepted path (C ABI ``spec_kv_commit_path``), in
    place.  ``cache``: contiguous CUDA tensor [planes, B, L, ...] (one entry =
    the trailing dimensions of one position)."""
    torch = _torch()
    planes, B, L = cache.shape[:3]
    entry = cache[0, 0, 0].numel() * cache.element_size()
    st = load_library().spec_kv_commit_path(
        _dev(cache, "cache"), B, planes, B * L * entry, L * entry, entry, L, int(N),
        _dev(base_len, "base_len", torch.int32), _dev(accepted_len, "accepted_len", torch.int32),
        _dev(path_nodes, "path_nodes", torch.int32), path_nodes.shape[1] - 1,
        _dev(new_len, "new_len", torch.int32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_kv_commit_path")


def spec_lm_head_verify_greedy(hidden, w_lm, draft_tokens, accepted_len, out_tokens, workspace,
                               stream=None):
    """LM head fused with greedy verification (C ABI
    ``spec_lm_head_verify_greedy``): ``hidden`` bf16 [B*(k+1), d], ``w_lm``
    bf16 [V, d], ``draft_tokens`` int32 [B, k]."""
    torch = _torch()
    B, k = draft_tokens.shape
    rows, d = hidden.shape
    V = w_lm.shape[0]
    if rows != B * (k + 1) or w_lm.shape[1] != d:
        raise ValueError("hidden must be [B*(k+1), d] and w_lm [V, d]")
    st = load_library().spec_lm_head_verify_greedy(
        _dev(hidden, "hidden", torch.bfloat16), _dev(w_lm, "w_lm", torch.bfloat16),
        _dev(draft_tokens, "draft_tokens", torch.int32), B, k, d, V,
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_lm_head_verify_greedy")


def spec_lm_head_verify_sample(h_target, h_draft, w_lm, draft_tokens, u_accept, u_sample,
                               temperature, accepted_len, out_tokens, p_out, q_out, resid_mass,
                               workspace, stream=None):
    """LM head fused with sampling verification (C ABI
    ``spec_lm_head_verify_sample``): ``h_target`` bf16 [B*(k+1), d],
    ``h_draft`` bf16 [B*k, d], ``w_lm`` bf16 [V, d], the rest as
    :func:`spec_verify_sample`."""
    torch = _torch()
    B, k = draft_tokens.shape
    rows, d = h_target.shape
    V = w_lm.shape[0]
    if rows != B * (k + 1) or w_lm.shape[1] != d:
        raise ValueError("h_target must be [B*(k+1), d] and w_lm [V, d]")
    if k > 0 and tuple(h_draft.shape) != (B * k, d):
        raise ValueError("h_draft must be [B*k, d]")
    st = load_library().spec_lm_head_verify_sample(
        _dev(h_target, "h_target", torch.bfloat16),
        _dev(h_draft, "h_draft", torch.bfloat16, optional=k == 0),
        _dev(w_lm, "w_lm", torch.bfloat16),
        _dev(draft_tokens, "draft_tokens", torch.int32, optional=k == 0),
        _dev(u_accept, "u_accept", torch.float32, optional=k == 0),
        _dev(u_sample, "u_sample", torch.float32), float(temperature), B, k, d, V,
        _dev(accepted_len, "accepted_len", torch.int32),
        _dev(out_tokens, "out_tokens", torch.int32),
        _dev(p_out, "p_out", torch.float32, optional=k == 0),
        _dev(q_out, "q_out", torch.float32, optional=k == 0),
        _dev(resid_mass, "resid_mass", torch.float32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_lm_head_verify_sample")


def spec_tree_grow(draft_logits, temperature, M, tokens, parents, depth, values, workspace,
                   stream=None):
    """EAGLE-2 tree growth (C ABI ``spec_tree_grow``): ``draft_logits``
    [B, D, K, V] bf16 or fp32; outputs [B, M+1]."""
    torch = _torch()
    B, D, K, V = draft_logits.shape
    st = load_library().spec_tree_grow(
        _dev(draft_logits, "draft_logits"), _dtype_code(draft_logits), float(temperature),
        B, D, K, V, int(M), _dev(tokens, "tokens", torch.int32),
        _dev(parents, "parents", torch.int32), _dev(depth, "depth", torch.int32),
        _dev(values, "values", torch.float32),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream))
    _check(st, "spec_tree_grow")


def spec_verify_tree_sample(target_logits, node_tokens, parents, u_sample, temperature, max_depth,
                            accepted_len, path_nodes, out_tokens, out_probs, workspace,
                            stream=None):
    """Sampling verification of draft trees (C ABI ``spec_verify_tree_sample``).

    target_logits [B, N, V] (bf16 or fp32); node_tokens, parents int32 [B, N];
    u_sample float32 [B, max_depth+1].  Outputs: accepted_len int32 [B];
    path_nodes, out_tokens int32 and out_probs float32 [B, max_depth+1].
    """
    torch = _torch()
    dev = _call_device(target_logits, "target_logits")
    B, N, V = target_logits.shape
    W = int(max_depth) + 1
    i32, f32 = torch.int32, torch.float32
    st = load_library().spec_verify_tree_sample(
        _dev(target_logits, "target_logits"), _dtype_code(target_logits),
        _arg(node_tokens, "node_tokens", i32, (B, N), dev),
        _arg(parents, "parents", i32, (B, N), dev), _arg(u_sample, "u_sample", f32, (B, W), dev),
        float(temperature), B, N, V, W - 1, _arg(accepted_len, "accepted_len", i32, (B,), dev),
        _arg(path_nodes, "path_nodes", i32, (B, W), dev),
        _arg(out_tokens, "out_tokens", i32, (B, W), dev),
        _arg(out_probs, "out_probs", f32, (B, W), dev), *_workspace(workspace, dev),
        _stream_of(stream, dev))
    _check(st, "spec_verify_tree_sample")


def spec_tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, base_len, depth, q_out, k_cache,
                       v_cache, workspace, pos_offset=0, interleaved=False, stream=None):
    """Head norms, rotation and cache write of the tree's nodes (C ABI
    ``spec_tree_qkv_rope``).

    qkv bf16 [B, N, Hq + 2 Hkv, D]; q_norm, k_norm bf16 [D] or None; inv_freq
    float32 [rot_dim / 2] or None (no rotation); base_len int32 [B]; depth int32 [B, N] or None (a
    chain); q_out bf16 [B, N, Hq, D]; k_cache, v_cache bf16 [B, L, Hkv, D],
    written at positions base_len - 1 + node.
    """
    torch = _torch()
    dev = _call_device(qkv, "qkv")
    B, N, H, D = qkv.shape
    Hkv = k_cache.shape[2] if k_cache.dim() == 4 else 0
    Hq = H - 2 * Hkv
    bf16 = torch.bfloat16
    kp, vp, stride, L = _cache_args(k_cache, v_cache, Hkv, D, B, dev)
    st = load_library().spec_tree_qkv_rope(
        _arg(qkv, "qkv", bf16, (B, N, H, D), dev),
        None if q_norm is None else _arg(q_norm, "q_norm", bf16, (D,), dev),
        None if k_norm is None else _arg(k_norm, "k_norm", bf16, (D,), dev), float(eps),
        None if inv_freq is None else _arg(inv_freq, "inv_freq", torch.float32,
                                           (inv_freq.numel(),), dev),
        0 if inv_freq is None else 2 * inv_freq.numel(),
        1 if interleaved else 0, int(pos_offset),
        _arg(base_len, "base_len", torch.int32, (B,), dev),
        None if depth is None else _arg(depth, "depth", torch.int32, (B, N), dev), B, N, Hq, Hkv,
        D, L, stride, _arg(q_out, "q_out", bf16, (B, N, Hq, D), dev), kp, vp,
        *_workspace(workspace, dev), _stream_of(stream, dev))
    _check(st, "spec_tree_qkv_rope")


def spec_tree_attention_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, D: int,
                                        P: int = 0) -> int:
    return int(load_library().spec_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, P))


def spec_tree_attention(q, k_cache, v_cache, mask, base_len, scale, out, lse, workspace,
                        prefix_k=None, prefix_v=None, stream=None):
    """Attention of the tree's nodes (C ABI ``spec_tree_attention``).

    q, out bf16 [B, N, Hq, D]; k_cache, v_cache bf16 [B, L, Hkv, D]; mask
    int32 [B, N, ceil(N/32)] (:func:`tree_attention_mask`) or None for a
    chain; base_len int32 [B]; lse float32 [B, N, Hq] or None; prefix_k,
    prefix_v bf16 [P, Hkv, D], a prefix that the whole batch shares, or None.
    """
    torch = _torch()
    dev = _call_device(q, "q")
    B, N, Hq, D = q.shape
    Hkv = k_cache.shape[2] if k_cache.dim() == 4 else 0
    bf16 = torch.bfloat16
    kp, vp, stride, L = _cache_args(k_cache, v_cache, Hkv, D, B, dev)
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError("prefix_k and prefix_v go together")
    P = 0 if prefix_k is None else prefix_k.shape[0]
    st = load_library().spec_tree_attention(
        _arg(q, "q", bf16, (B, N, Hq, D), dev), kp, vp, stride, L,
        _arg(prefix_k, "prefix_k", bf16, (P, Hkv, D), dev) if P else None,
        _arg(prefix_v, "prefix_v", bf16, (P, Hkv, D), dev) if P else None, P,
        None if mask is None else _arg(mask, "mask", torch.int32, (B, N, (N + 31) // 32), dev),
        _arg(base_len, "base_len", torch.int32, (B,), dev), B, N, Hq, Hkv, D, float(scale),
        _arg(out, "out", bf16, (B, N, Hq, D), dev),
        None if lse is None else _arg(lse, "lse", torch.float32, (B, N, Hq), dev),
        *_workspace(workspace, dev), _stream_of(stream, dev))
    _check(st, "spec_tree_attention")


def spec_verify_read_flags(workspace, clear: bool = True, stream=None) -> int:
    """Device flag bits recorded in ``workspace`` (synchronises the stream)."""
    out = ctypes.c_uint32(0)
    st = load_library().spec_verify_read_flags(_dev(workspace, "workspace"), ctypes.byref(out),
                                               1 if clear else 0, _stream_ptr(stream))
    _check(st, "spec_verify_read_flags")
    return int(out.value)


# ---------------------------------------------------------------------------
# convenience: allocate outputs + workspace with torch, then call the C ABI
# ---------------------------------------------------------------------------

def alloc_workspace(mode: int, B: int, k_or_N: int, V: int, dtype: int, device="cuda"):
    """Zero-filled workspace for one call shape (reusable for any smaller one)."""
    n = spec_verify_workspace_bytes(mode, B, k_or_N, V, dtype)
    if n == 0:
        raise ValueError("shape outside the library's limits")
    return _torch().zeros(n, dtype=_torch().uint8, device=device)


def verify_sample(target_logits, draft_logits, draft_tokens, u_accept, u_sample, temperature,
                  workspace=None, stream=None):
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = target_logits.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_SAMPLE, B, k, V, _dtype_code(target_logits), dev)
    out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
               out_tokens=torch.empty(B, k + 1, dtype=torch.int32, device=dev),
               p=torch.empty(B, k, dtype=torch.float32, device=dev),
               q=torch.empty(B, k, dtype=torch.float32, device=dev),
               resid_mass=torch.empty(B, dtype=torch.float32, device=dev))
    spec_verify_sample(target_logits, draft_logits, draft_tokens, u_accept, u_sample,
                       temperature, out["accepted_len"], out["out_tokens"], out["p"], out["q"],
                       out["resid_mass"], workspace, stream)
    return out


def verify_greedy(target_logits, draft_tokens, workspace=None, stream=None):
    torch = _torch()
    B, k1, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_GREEDY, B, k1 - 1, V, _dtype_code(target_logits),
                                    dev)
    out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
               out_tokens=torch.empty(B, k1, dtype=torch.int32, device=dev))
    spec_verify_greedy(target_logits, draft_tokens, out["accepted_len"], out["out_tokens"],
                       workspace, stream)
    return out


def verify_tree_greedy(target_logits, node_tokens, parents, max_depth, workspace=None,
                       stream=None):
    torch = _torch()
    B, N, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_TREE_GREEDY, B, N, V,
                                    _dtype_code(target_logits), dev)
    W = int(max_depth) + 1
    out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
               path_nodes=torch.empty(B, W, dtype=torch.int32, device=dev),
               out_tokens=torch.empty(B, W, dtype=torch.int32, device=dev))
    spec_verify_tree_greedy(target_logits, node_tokens, parents, max_depth,
                            out["accepted_len"], out["path_nodes"], out["out_tokens"],
                            workspace, stream)
    return out


def tree_attention_mask(parents, workspace=None, stream=None):
    """Ancestor bitmask and depth of B draft trees: returns ``(mask, depth)``
    with mask int32 [B, N, ceil(N/32)] (the bit patterns of the C ABI's
    uint32 words) and depth int32 [B, N]."""
    torch = _torch()
    B, N = parents.shape
    dev = parents.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_TREE_MASK, B, N, 1, SPEC_DTYPE_F32, dev)
    mask = torch.empty(B, N, (N + 31) // 32, dtype=torch.int32, device=dev)
    depth = torch.empty(B, N, dtype=torch.int32, device=dev)
    spec_tree_attention_mask(parents, mask, depth, workspace, stream)
    return mask, depth


def lm_head_verify_greedy(hidden, w_lm, draft_tokens, workspace=None, stream=None):
    """Greedy verification straight from hidden states and the LM head."""
    torch = _torch()
    B, k = draft_tokens.shape
    dev = hidden.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_LM_HEAD_GREEDY, B, k, w_lm.shape[0],
                                    SPEC_DTYPE_BF16, dev)
    out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
               out_tokens=torch.empty(B, k + 1, dtype=torch.int32, device=dev))
    spec_lm_head_verify_greedy(hidden, w_lm, draft_tokens, out["accepted_len"],
                               out["out_tokens"], workspace, stream)
    return out


def lm_head_verify_sample(h_target, h_draft, w_lm, draft_tokens, u_accept, u_sample, temperature,
                          workspace=None, stream=None):
    """Sampling verification straight from hidden states, drafted features
    and the LM head; returns the outputs of :func:`verify_sample`."""
    torch = _torch()
    B, k = draft_tokens.shape
    dev = h_target.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_LM_HEAD_SAMPLE, B, k, w_lm.shape[0],
                                    SPEC_DTYPE_BF16, dev)
    i32 = dict(dtype=torch.int32, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(accepted_len=torch.empty(B, **i32), out_tokens=torch.empty(B, k + 1, **i32),
               p=torch.empty(B, k, **f32), q=torch.empty(B, k, **f32),
               resid_mass=torch.empty(B, **f32))
    spec_lm_head_verify_sample(h_target, h_draft, w_lm, draft_tokens, u_accept, u_sample,
                               temperature, out["accepted_len"], out["out_tokens"], out["p"],
                               out["q"], out["resid_mass"], workspace, stream)
    return out


def tree_grow(draft_logits, temperature, M, workspace=None, stream=None):
    """Grow B draft trees; returns dict(tokens, parents, depth, values) [B, M+1]."""
    torch = _torch()
    B, D, K, V = draft_logits.shape
    dev = draft_logits.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_TREE_GROW, B, K, V, _dtype_code(draft_logits), dev)
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(tokens=torch.empty(B, M + 1, **i32), parents=torch.empty(B, M + 1, **i32),
               depth=torch.empty(B, M + 1, **i32),
               values=torch.empty(B, M + 1, dtype=torch.float32, device=dev))
    spec_tree_grow(draft_logits, temperature, M, out["tokens"], out["parents"], out["depth"],
                   out["values"], workspace, stream)
    return out


def _allocating_on(stream, device):
    """Context in which what a convenience allocates belongs to the stream that
    its call runs on: the allocator then hands a workspace that goes out of use
    to that stream's later work only."""
    cuda = _torch().cuda
    if isinstance(stream, int):
        stream = cuda.ExternalStream(stream, device=device) if stream else cuda.default_stream(device)
    return cuda.stream(stream)


def verify_tree_sample(target_logits, node_tokens, parents, u_sample, temperature, max_depth,
                       workspace=None, stream=None):
    """Sampling verification of B draft trees; returns dict(accepted_len,
    path_nodes, out_tokens, out_probs)."""
    if stream is not None:
        with _allocating_on(stream, target_logits.device):
            return verify_tree_sample(target_logits, node_tokens, parents, u_sample, temperature,
                                      max_depth, workspace)
    torch = _torch()
    B, N, V = target_logits.shape
    dev = target_logits.device
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_TREE_SAMPLE, B, N, V, _dtype_code(target_logits),
                                    dev)
    W = int(max_depth) + 1
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(accepted_len=torch.empty(B, **i32), path_nodes=torch.empty(B, W, **i32),
               out_tokens=torch.empty(B, W, **i32),
               out_probs=torch.empty(B, W, dtype=torch.float32, device=dev))
    spec_verify_tree_sample(target_logits, node_tokens, parents, u_sample, temperature, max_depth,
                            out["accepted_len"], out["path_nodes"], out["out_tokens"],
                            out["out_probs"], workspace, stream)
    return out


def tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, base_len, depth, k_cache, v_cache,
                  pos_offset=0, interleaved=False, workspace=None, stream=None):
    """Normalise and rotate the tree's query and key heads and write its keys
    and values into the cache; returns the queries [B, N, Hq, D]."""
    if stream is not None:
        with _allocating_on(stream, qkv.device):
            return tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, base_len, depth, k_cache,
                                 v_cache, pos_offset, interleaved, workspace)
    torch = _torch()
    B, N, H, D = qkv.shape
    Hq = H - 2 * _cache_heads(k_cache)
    if Hq < 1:
        raise ValueError(f"qkv holds {H} heads, of which {H - Hq} are keys and values: no query head")
    if workspace is None:
        workspace = alloc_workspace(SPEC_MODE_TREE_QKV, B, N, 1, SPEC_DTYPE_BF16, qkv.device)
    q = torch.empty(B, N, Hq, D, dtype=qkv.dtype, device=qkv.device)
    spec_tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, base_len, depth, q, k_cache, v_cache,
                       workspace, pos_offset, interleaved, stream)
    return q


def alloc_tree_attention_workspace(q, k_cache, prefix_k=None):
    """Workspace of :func:`spec_tree_attention` for these shapes (its flag word
    is zero; the rest needs no value)."""
    torch = _torch()
    B, N, Hq, D = q.shape
    n = spec_tree_attention_workspace_bytes(B, N, Hq, _cache_heads(k_cache), D,
                                            0 if prefix_k is None else prefix_k.shape[0])
    if n == 0:
        raise ValueError("shape outside the library's limits")
    ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    ws[:256].zero_()
    return ws


def tree_attention(q, k_cache, v_cache, mask, base_len, scale=None, prefix_k=None, prefix_v=None,
                   workspace=None, stream=None):
    """Attention of the tree's nodes over a shared prefix, the cached positions
    and their ancestors; returns ``(out, lse)``.  ``scale`` defaults to
    1 / sqrt(D)."""
    if stream is not None:
        with _allocating_on(stream, q.device):
            return tree_attention(q, k_cache, v_cache, mask, base_len, scale, prefix_k, prefix_v,
                                  workspace)
    torch = _torch()
    if workspace is None:
        workspace = alloc_tree_attention_workspace(q, k_cache, prefix_k)
    if scale is None:
        scale = q.shape[3] ** -0.5
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    spec_tree_attention(q, k_cache, v_cache, mask, base_len, scale, out, lse, workspace,
                        prefix_k, prefix_v, stream)
    return out, lse


def to_device_logits(arr, dtype: str, device="cuda"):
    """numpy logits (float32, or uint16 bf16 bits) -> torch CUDA tensor."""
    import numpy as np
    torch = _torch()
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr, dtype=np.float32))
    return t.to(device)
