"""Thin Python binding of librapid.so (argument marshalling only).

Every step of the verification path runs in the CUDA kernels behind the C
ABI declared in include/rapid.h; this module only turns torch tensors into
device pointers, sizes workspaces and passes the current CUDA stream.  There
is no CPU or PyTorch fallback: if librapid.so is missing or cannot be loaded,
every call raises.
"""
import contextlib
import ctypes
import functools
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "librapid.so")

RAPID_OK = 0
RAPID_EINVAL = -1
RAPID_ECUDA = -2
RAPID_ENOMEM = -3
RAPID_ETIMEOUT = -4
RAPID_EUNSUPPORTED = -5
RAPID_DTYPE_F32 = 0
RAPID_DTYPE_BF16 = 1
RAPID_ACCEPT_TAIL_CLAMP = 1
RAPID_MAX_NQ = 64
RAPID_MAX_VOCAB = 229376
RAPID_COMMIT_MAX_LAYERS = 128
RAPID_RETRIEVAL_MAX_CHUNKS = 8192
RAPID_LM_HEAD_MAX_ROWS = 256
RAPID_NOALLOC_MAX_NODES = 4096
RAPID_ROPE_INTERLEAVED = 1
RAPID_Q8_PAGE_TOKENS = 64
RAPID_Q8_MAX_PAGES = 1 << 24

_lib = None


class RapidError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """Load librapid.so (built by __graft_entry__.build()); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RapidError(f"librapid.so is not built ({LIB_PATH} missing); "
                         "run `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, u32, u64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                       ctypes.c_float, ctypes.c_uint32, ctypes.c_uint64,
                                       ctypes.c_size_t)
    L.rapid_verify_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, i32]
    L.rapid_verify_attn_workspace_size.restype = sz
    L.rapid_verify_attn.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i64, vp, vp, f32,
                                    vp, vp, vp, sz, vp]
    L.rapid_verify_attn.restype = i32
    L.rapid_attn_merge.argtypes = [vp, vp, i32, i32, i64, i32, vp, vp, vp]
    L.rapid_attn_merge.restype = i32
    L.rapid_accept_workspace_size.argtypes = [i32, i32, i32]
    L.rapid_accept_workspace_size.restype = sz
    L.rapid_accept.argtypes = [vp, vp, vp, vp, i32, i32, i32, f32, f32, u64, u32, vp, vp, vp, vp,
                               vp, sz, vp]
    L.rapid_accept.restype = i32
    L.rapid_accept_ex.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, f32, f32, u64, vp, u32, vp,
                                  vp, vp, vp, vp, sz, vp]
    L.rapid_accept_ex.restype = i32
    L.rapid_status_string.argtypes = [i32]
    L.rapid_status_string.restype = ctypes.c_char_p
    L.rapid_version.argtypes = []
    L.rapid_version.restype = i32
    L.rapid_device_error.argtypes = [i32]
    L.rapid_device_error.restype = i32
    L.rapid_device_error_info.argtypes = [vp, i32]
    L.rapid_device_error_info.restype = i32
    L.rapid_stream_status.argtypes = [vp, i32]
    L.rapid_stream_status.restype = i32
    L.rapid_wait_selftest.argtypes = [u64, vp]
    L.rapid_wait_selftest.restype = i32
    L.rapid_accept_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, f32, f32, u64, u32, vp, vp,
                                       vp, vp, vp]
    L.rapid_accept_noalloc.restype = i32
    L.rapid_kv_commit.argtypes = [vp, vp, i32, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp]
    L.rapid_kv_commit.restype = i32
    L.rapid_kv_advance.argtypes = [vp, vp, i32, i32, i64, vp]
    L.rapid_kv_advance.restype = i32
    L.rapid_retrieval_scores.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp]
    L.rapid_retrieval_scores.restype = i32
    L.rapid_retrieval_select.argtypes = [vp, vp, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp]
    L.rapid_retrieval_select.restype = i32
    L.rapid_lm_head.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    L.rapid_lm_head.restype = i32
    L.rapid_lm_head_accept_workspace_size.argtypes = [i32, i32, i32]
    L.rapid_lm_head_accept_workspace_size.restype = ctypes.c_size_t
    L.rapid_lm_head_accept.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, f32, u64, u32,
                                       vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.rapid_lm_head_accept.restype = i32
    L.rapid_lm_head_accept_ex.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, f32, f32,
                                          u64, vp, u32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.rapid_lm_head_accept_ex.restype = i32
    L.rapid_qkv_append.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, f32, vp,
                                   i32, u32, vp, vp, vp, vp, vp, vp, vp, i64, vp]
    L.rapid_qkv_append.restype = i32
    L.rapid_kv_seal.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i32, i32, vp, i32,
                                vp, vp, vp]
    L.rapid_kv_seal.restype = i32
    L.rapid_kv_seal_advance.argtypes = [vp, vp, vp, i32, i32, i32, i64, i32, vp]
    L.rapid_kv_seal_advance.restype = i32
    L.rapid_verify_attn_q8_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, i32, i32]
    L.rapid_verify_attn_q8_workspace_size.restype = sz
    L.rapid_verify_attn_q8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64,
                                       i32, i32, vp, vp, vp, f32, vp, vp, vp, sz, vp]
    L.rapid_verify_attn_q8.restype = i32
    _lib = L
    return L


def _check(status: int, what: str):
    if status != RAPID_OK:
        msg = lib().rapid_status_string(status).decode()
        raise RapidError(f"{what} failed: {msg} ({status})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise RapidError("librapid works on CUDA tensors only (no CPU path)")
        if t is not None and not t.is_contiguous():
            raise RapidError("librapid needs contiguous tensors")


def _need_same_device(*ts):
    """Every tensor on the current CUDA device (the launches go to it)."""
    cur = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.device.index != cur:
            raise RapidError(f"tensor on {t.device}, but the current device is cuda:{cur}")


def _need(t, dtype, shape, name):
    if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape)):
        raise RapidError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _refuse(t, dev, dtype, shape, name):
    """The reason why _arg turned a tensor away."""
    if not isinstance(t, torch.Tensor):
        raise RapidError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise RapidError(f"{name}: librapid works on CUDA tensors only (no CPU path)")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise RapidError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise RapidError(f"{name}: librapid needs contiguous tensors")
    raise RapidError(f"{name} is on {t.device}, but the current device is cuda:{dev}")


def _arg(t, dev, dtype, shape, name):
    """The address of a contiguous tensor of this type and shape on device `dev` (one test
    of each, a few hundred nanoseconds: a short kernel waits for the host)."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _refuse(t, dev, dtype, shape, name)
    return t.data_ptr()


def _device_of(t, name):
    """The current device, which `t` has to be on."""
    dev = t.get_device()
    if dev < 0:
        raise RapidError(f"{name}: librapid works on CUDA tensors only (no CPU path)")
    cur = torch.cuda.current_device()
    if dev != cur:
        raise RapidError(f"{name} is on {t.device}, but the current device is cuda:{cur}")
    return dev


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _check_accept_tensors(z_target, q_draft, draft_tokens, parent, n_accepted, next_token, path,
                          diag, n_nodes=None):
    """The sizes the kernels will index by: z and q float32 [B, n_q, V]; tokens,
    parents and the path int32 [B, n_q]; counts int32 [B]; diag float32 [B, n_q, 5]."""
    if z_target is None or z_target.dim() != 3:
        raise RapidError("z_target must be a [B, n_q, V] tensor")
    B, n_q, V = z_target.shape
    _need(z_target, torch.float32, (B, n_q, V), "z_target")
    _need(q_draft, torch.float32, (B, n_q, V), "q_draft")
    _need(draft_tokens, torch.int32, (B, n_q), "draft_tokens")
    _need(parent, torch.int32, (B, n_q), "parent")
    _need(n_accepted, torch.int32, (B,), "n_accepted")
    _need(next_token, torch.int32, (B,), "next_token")
    _need(path, torch.int32, (B, n_q), "path")
    _need(diag, torch.float32, (B, n_q, 5), "diag")
    _need(n_nodes, torch.int32, (B,), "n_nodes")
    _need_same_device(z_target, q_draft, draft_tokens, parent, n_accepted, next_token, path, diag,
                      n_nodes)
    return B, n_q, V


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RAPID_DTYPE_BF16
    if t.dtype == torch.float32:
        return RAPID_DTYPE_F32
    raise RapidError(f"unsupported dtype {t.dtype}")


# ---------------------------------------------------------------------------
# C-ABI mirrors (same names, same argument order; tensors in place of pointers)
# ---------------------------------------------------------------------------

def rapid_verify_attn_workspace_size(B, Hq, Hkv, d, n_q, kv_capacity, dtype) -> int:
    return int(lib().rapid_verify_attn_workspace_size(B, Hq, Hkv, d, n_q, kv_capacity, dtype))


def rapid_verify_attn(Q, Kcache, Vcache, prefix_len, spec_mask, softmax_scale, O, LSE,
                      workspace, stream=None):
    """Launch verify attention; shapes are read from the tensors."""
    _need_cuda(Q, Kcache, Vcache, prefix_len, spec_mask, O, LSE, workspace)
    B, Hq, n_q, d = Q.shape
    Hkv, cap = Kcache.shape[1], Kcache.shape[2]
    st = lib().rapid_verify_attn(_ptr(Q), _ptr(Kcache), _ptr(Vcache), _dtype_code(Q), B, Hq, Hkv,
                                 d, n_q, cap, _ptr(prefix_len), _ptr(spec_mask),
                                 float(softmax_scale), _ptr(O), _ptr(LSE), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "rapid_verify_attn")


def rapid_attn_merge(O_parts, LSE_parts, O, LSE, stream=None):
    """Log-sum-exp merge of n_parts attention results: O_parts [n_parts, ..., d] (bf16 or
    fp32), LSE_parts [n_parts, ...] float32 -> O [..., d], LSE [...]."""
    _need_cuda(O_parts, LSE_parts, O, LSE)
    n_parts, d = O_parts.shape[0], O_parts.shape[-1]
    rows = LSE_parts[0].numel()
    if (LSE_parts.dtype != torch.float32 or LSE.dtype != torch.float32 or O.dtype != O_parts.dtype
            or O_parts.numel() != n_parts * rows * d or O.numel() != rows * d
            or LSE.numel() != rows):
        raise RapidError("rapid_attn_merge: mismatched shapes or dtypes")
    st = lib().rapid_attn_merge(_ptr(O_parts), _ptr(LSE_parts), _dtype_code(O_parts), n_parts,
                                rows, d, _ptr(O), _ptr(LSE), _stream(stream))
    _check(st, "rapid_attn_merge")


def rapid_accept_workspace_size(B, n_q, V) -> int:
    return int(lib().rapid_accept_workspace_size(B, n_q, V))


def rapid_accept(z_target, q_draft, draft_tokens, parent, T, eta, philox_seed, flags,
                 n_accepted, next_token, path, diag, workspace, stream=None):
    _need_cuda(z_target, q_draft, draft_tokens, parent, n_accepted, next_token, path, diag,
               workspace)
    B, n_q, V = _check_accept_tensors(z_target, q_draft, draft_tokens, parent, n_accepted,
                                      next_token, path, diag)
    st = lib().rapid_accept(_ptr(z_target), _ptr(q_draft), _ptr(draft_tokens), _ptr(parent), B,
                            n_q, V, float(T), float(eta), int(philox_seed) & ((1 << 64) - 1),
                            int(flags), _ptr(n_accepted), _ptr(next_token), _ptr(path),
                            _ptr(diag), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "rapid_accept")


def rapid_accept_ex(z_target, q_draft, draft_tokens, parent, n_nodes, T, eta, philox_seed,
                    flags, n_accepted, next_token, path, diag, workspace, stream=None):
    """rapid_accept with optional per-sequence node counts n_nodes (int32 [B] CUDA tensor or
    None) and a Philox key that is either an int or a one-element 64-bit integer CUDA tensor
    read by the kernels when they run."""
    _need_cuda(z_target, q_draft, draft_tokens, parent, n_nodes, n_accepted, next_token, path,
               diag, workspace)
    B, n_q, V = _check_accept_tensors(z_target, q_draft, draft_tokens, parent, n_accepted,
                                      next_token, path, diag, n_nodes)
    if isinstance(philox_seed, torch.Tensor):
        _need_cuda(philox_seed)
        if philox_seed.dtype not in (torch.int64, torch.uint64) or philox_seed.numel() != 1:
            raise RapidError("a device philox_seed must be a one-element 64-bit integer tensor")
        key, key_dev = 0, _ptr(philox_seed)
    else:
        key, key_dev = int(philox_seed) & ((1 << 64) - 1), None
    st = lib().rapid_accept_ex(_ptr(z_target), _ptr(q_draft), _ptr(draft_tokens), _ptr(parent),
                               _ptr(n_nodes), B, n_q, V, float(T), float(eta), key, key_dev,
                               int(flags), _ptr(n_accepted), _ptr(next_token), _ptr(path),
                               _ptr(diag), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "rapid_accept_ex")


def rapid_accept_noalloc(z_target, q_draft, draft_tokens, parent, T, eta, philox_seed, flags,
                         n_accepted, next_token, path, diag, stream=None):
    """rapid_accept with the library's static scratch instead of a workspace."""
    _need_cuda(z_target, q_draft, draft_tokens, parent, n_accepted, next_token, path, diag)
    B, n_q, V = _check_accept_tensors(z_target, q_draft, draft_tokens, parent, n_accepted,
                                      next_token, path, diag)
    st = lib().rapid_accept_noalloc(_ptr(z_target), _ptr(q_draft), _ptr(draft_tokens),
                                    _ptr(parent), B, n_q, V, float(T), float(eta),
                                    int(philox_seed) & ((1 << 64) - 1), int(flags),
                                    _ptr(n_accepted), _ptr(next_token), _ptr(path), _ptr(diag),
                                    _stream(stream))
    _check(st, "rapid_accept_noalloc")


def rapid_lm_head(hidden, W_lm, z, stream=None):
    """Logits z [rows, V] (fp32) of hidden [rows, hidden_dim] against W_lm [V, hidden_dim] (bf16)."""
    _need_cuda(hidden, W_lm, z)
    rows, hd = hidden.shape
    V = W_lm.shape[0]
    _need(hidden, torch.bfloat16, (rows, hd), "hidden")
    _need(W_lm, torch.bfloat16, (V, hd), "W_lm")
    _need(z, torch.float32, (rows, V), "z")
    _need_same_device(hidden, W_lm, z)
    st = lib().rapid_lm_head(_ptr(hidden), _ptr(W_lm), rows, hd, V, _ptr(z), _stream(stream))
    _check(st, "rapid_lm_head")


def rapid_lm_head_accept_workspace_size(B, n_q, V):
    return int(lib().rapid_lm_head_accept_workspace_size(B, n_q, V))


def rapid_lm_head_accept(hidden, W_lm, q_draft, draft_tokens, parent, T, eta, philox_seed, flags,
                         n_accepted, next_token, path, diag, workspace, stream=None):
    """rapid_accept on the logits of hidden [B*n_q, hidden_dim] against W_lm [V, hidden_dim]."""
    _need_cuda(hidden, W_lm, q_draft, draft_tokens, parent, n_accepted, next_token, path, diag,
               workspace)
    B, n_q, V = _check_accept_tensors(q_draft, q_draft, draft_tokens, parent, n_accepted,
                                      next_token, path, diag)
    _need(hidden, torch.bfloat16, (B * n_q, hidden.shape[-1]), "hidden")
    _need(W_lm, torch.bfloat16, (V, hidden.shape[-1]), "W_lm")
    _need_same_device(hidden, W_lm, workspace)
    st = lib().rapid_lm_head_accept(_ptr(hidden), _ptr(W_lm), hidden.shape[1], _ptr(q_draft),
                                    _ptr(draft_tokens), _ptr(parent), B, n_q, V, float(T),
                                    float(eta), int(philox_seed) & ((1 << 64) - 1), int(flags),
                                    _ptr(n_accepted), _ptr(next_token), _ptr(path), _ptr(diag),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check(st, "rapid_lm_head_accept")


def rapid_lm_head_accept_ex(hidden, W_lm, q_draft, draft_tokens, parent, n_nodes, T, eta,
                            philox_seed, flags, n_accepted, next_token, path, diag, workspace,
                            stream=None):
    """rapid_lm_head_accept with rapid_accept_ex's node counts and device Philox key
    (philox_seed: an int, or a one-element 64-bit integer CUDA tensor)."""
    _need_cuda(hidden, W_lm, q_draft, draft_tokens, parent, n_nodes, n_accepted, next_token,
               path, diag, workspace)
    B, n_q, V = _check_accept_tensors(q_draft, q_draft, draft_tokens, parent, n_accepted,
                                      next_token, path, diag, n_nodes)
    _need(hidden, torch.bfloat16, (B * n_q, hidden.shape[-1]), "hidden")
    _need(W_lm, torch.bfloat16, (V, hidden.shape[-1]), "W_lm")
    _need_same_device(hidden, W_lm, workspace)
    if isinstance(philox_seed, torch.Tensor):
        _need_cuda(philox_seed)
        if philox_seed.dtype not in (torch.int64, torch.uint64) or philox_seed.numel() != 1:
            raise RapidError("a device philox_seed must be a one-element 64-bit integer tensor")
        key, key_dev = 0, _ptr(philox_seed)
    else:
        key, key_dev = int(philox_seed) & ((1 << 64) - 1), None
    st = lib().rapid_lm_head_accept_ex(_ptr(hidden), _ptr(W_lm), hidden.shape[1], _ptr(q_draft),
                                       _ptr(draft_tokens), _ptr(parent), _ptr(n_nodes), B, n_q,
                                       V, float(T), float(eta), key, key_dev, int(flags),
                                       _ptr(n_accepted), _ptr(next_token), _ptr(path),
                                       _ptr(diag), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream))
    _check(st, "rapid_lm_head_accept_ex")


class KVLayerTable:
    """The device addresses of every layer's K and V cache, checked and packed
    once, for repeated rapid_kv_commit calls on the same caches (the per-call
    packing of a few dozen pointers otherwise costs tens of microseconds of
    host time)."""

    def __init__(self, K_layers, V_layers):
        if len(K_layers) != len(V_layers) or not K_layers:
            raise RapidError("rapid_kv_commit needs matching, non-empty K and V layer lists")
        if len(K_layers) > RAPID_COMMIT_MAX_LAYERS:
            raise RapidError(f"at most {RAPID_COMMIT_MAX_LAYERS} layers per call")
        _need_cuda(*K_layers, *V_layers)
        shape, dtype = tuple(K_layers[0].shape), K_layers[0].dtype
        for t in list(K_layers) + list(V_layers):
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise RapidError("every layer's K and V cache needs the same shape and dtype")
        self.layers = len(K_layers)
        self.B, self.Hkv, self.cap, self.d = shape
        self.dtype = _dtype_code(K_layers[0])
        self._k = (ctypes.c_void_p * self.layers)(*[t.data_ptr() for t in K_layers])
        self._v = (ctypes.c_void_p * self.layers)(*[t.data_ptr() for t in V_layers])
        self._keep = (list(K_layers), list(V_layers))   # the caches outlive the table

    def commit(self, prefix_len, path, n_accepted, stream=None):
        st = lib().rapid_kv_commit(ctypes.cast(self._k, ctypes.c_void_p),
                                   ctypes.cast(self._v, ctypes.c_void_p), self.layers, self.dtype,
                                   self.B, self.Hkv, self.d, self.cap, path.shape[1],
                                   _ptr(prefix_len), _ptr(path), _ptr(n_accepted), _stream(stream))
        _check(st, "rapid_kv_commit")


def rapid_kv_commit(K_layers, V_layers, prefix_len, path, n_accepted, stream=None):
    """Move the accepted speculative K/V rows of every layer next to the root.

    K_layers, V_layers: sequences of [B, Hkv, kv_capacity, d] caches (one per
    layer), or K_layers a KVLayerTable and V_layers None; prefix_len [B],
    path [B, n_q], n_accepted [B] int32 on the device."""
    _need_cuda(prefix_len, path, n_accepted)
    table = K_layers if isinstance(K_layers, KVLayerTable) else KVLayerTable(K_layers, V_layers)
    table.commit(prefix_len, path, n_accepted, stream)


def rapid_kv_advance(prefix_len, n_accepted, n_q, kv_capacity, stream=None):
    """prefix_len += 1 + n_accepted (device, in place)."""
    _need_cuda(prefix_len, n_accepted)
    st = lib().rapid_kv_advance(_ptr(prefix_len), _ptr(n_accepted), prefix_len.shape[0], n_q,
                                kv_capacity, _stream(stream))
    _check(st, "rapid_kv_advance")


def rapid_retrieval_scores(query, chunks, scores, stream=None):
    """Cosine similarities scores [B, N] of chunks [B, N, D] with query [B, D]."""
    _need_cuda(query, chunks, scores)
    B, N, D = chunks.shape
    st = lib().rapid_retrieval_scores(_ptr(query), _ptr(chunks), _dtype_code(chunks), B, N, D,
                                      _ptr(scores), _stream(stream))
    _check(st, "rapid_retrieval_scores")


def rapid_retrieval_select(scores, context_tokens, selected, n_selected, tokens_selected,
                           chunk_tokens=512, threshold=0.3, min_tokens=4096, ratio=24, stream=None):
    """Kept chunk ids (ascending, then -1) per sequence under the RAG budget."""
    _need_cuda(scores, context_tokens, selected, n_selected, tokens_selected)
    B, N = scores.shape
    st = lib().rapid_retrieval_select(_ptr(scores), _ptr(context_tokens), B, N, chunk_tokens,
                                      float(threshold), min_tokens, ratio, _ptr(selected),
                                      _ptr(n_selected), _ptr(tokens_selected), _stream(stream))
    _check(st, "rapid_retrieval_select")


def _head_rows(t, dev, B, n, H, d, dtype, name):
    """Address, batch and token stride of projection rows [B, n, H, d] whose heads lie one
    after the other (a view of a fused projection will do)."""
    if t.shape != (B, n, H, d) or t.dtype != dtype or t.get_device() != dev:
        _refuse(t, dev, dtype, (B, n, H, d), name)
    sb, sn, sh, se = t.stride()
    if se != 1 or (H > 1 and sh != d):
        raise RapidError(f"{name}: the heads of a token must be contiguous")
    # the stride of a dimension of size 1 means nothing and may be anything
    return t.data_ptr(), (sb if B > 1 else 0), (sn if n > 1 else 0)


def rapid_qkv_append(q, k, v, q_weight, k_weight, eps, inv_freq, flags, prefix_len, pos_offset,
                     row_offset, n_rows, Q, Kcache, Vcache, stream=None):
    """Norm and rotate the rows q [B, n, Hq, d] and k [B, n, Hkv, d], write queries to
    Q [B, Hq, n, d] and keys and values to cache rows prefix_len + i; None for what is
    optional.  q, k and v may be views of one fused projection."""
    dev = _device_of(Q, "Q")
    if Q.dim() != 4 or Kcache.dim() != 4:
        raise RapidError("Q and the caches must have four dimensions")
    B, Hq, n, d = Q.shape
    Hkv, cap = Kcache.shape[1], Kcache.shape[2]
    dt = Q.dtype
    i32 = torch.int32
    q_ptr, qb, qt = _head_rows(q, dev, B, n, Hq, d, dt, "q")
    k_ptr, kb, kt = _head_rows(k, dev, B, n, Hkv, d, dt, "k")
    v_ptr, vb, vt = _head_rows(v, dev, B, n, Hkv, d, dt, "v")
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    st = lib().rapid_qkv_append(
        q_ptr, k_ptr, v_ptr, (ctypes.c_int64 * 6)(qb, qt, kb, kt, vb, vt), _dtype_code(Q), B, n,
        Hq, Hkv, d, _arg(q_weight, dev, dt, (d,), "q_weight"),
        _arg(k_weight, dev, dt, (d,), "k_weight"), eps,
        _arg(inv_freq, dev, torch.float32, (rot // 2,), "inv_freq"), rot, flags,
        _arg(prefix_len, dev, i32, (B,), "prefix_len"),
        _arg(pos_offset, dev, i32, (B,), "pos_offset"),
        _arg(row_offset, dev, i32, (B, n), "row_offset"), _arg(n_rows, dev, i32, (B,), "n_rows"),
        _arg(Q, dev, dt, (B, Hq, n, d), "Q"), _arg(Kcache, dev, dt, (B, Hkv, cap, d), "Kcache"),
        _arg(Vcache, dev, dt, (B, Hkv, cap, d), "Vcache"), cap, _raw_stream(stream, dev))
    _check(st, "rapid_qkv_append")


class Q8LayerTable:
    """The device addresses of every layer's tail caches [B, Hkv, tail_capacity, d], pages
    [n_pages, Hkv, 2, 64, d] (torch.float8_e4m3fn) and scales [n_pages, Hkv, 2] (float32),
    checked and packed once for repeated rapid_kv_seal calls."""

    def __init__(self, K_layers, V_layers, page_layers, scale_layers):
        lists = [list(x) for x in (K_layers, V_layers, page_layers, scale_layers)]
        if not lists[0] or len({len(x) for x in lists}) != 1:
            raise RapidError("rapid_kv_seal needs matching, non-empty layer lists")
        if len(lists[0]) > RAPID_COMMIT_MAX_LAYERS:
            raise RapidError(f"at most {RAPID_COMMIT_MAX_LAYERS} layers per call")
        for x in lists:
            _need_cuda(*x)
        K, V, pages, scales = lists
        if K[0].dim() != 4 or pages[0].dim() != 5:
            raise RapidError("tail caches are [B, Hkv, tail_capacity, d], pages [n_pages, Hkv, 2, 64, d]")
        self.layers = len(K)
        self.B, self.Hkv, self.cap, self.d = K[0].shape
        self.n_pages = pages[0].shape[0]
        self.dtype = _dtype_code(K[0])
        for t in K + V:
            _need(t, K[0].dtype, (self.B, self.Hkv, self.cap, self.d), "tail cache")
        for t in pages:
            _need(t, torch.float8_e4m3fn,
                  (self.n_pages, self.Hkv, 2, RAPID_Q8_PAGE_TOKENS, self.d), "pages")
        for t in scales:
            _need(t, torch.float32, (self.n_pages, self.Hkv, 2), "scales")
        _need_same_device(*K, *V, *pages, *scales)
        self.device = K[0].device
        self._ptrs = [(ctypes.c_void_p * self.layers)(*[t.data_ptr() for t in x]) for x in lists]
        self._keep = lists                                # the tensors outlive the table

    def _lengths(self, page_table, sealed_len, tail_len):
        dev = _device_of(self._keep[0][0], "tail cache")
        if page_table.dim() != 2:
            raise RapidError("page_table must be [B, max_pages]")
        max_pages, i32 = page_table.shape[1], torch.int32
        return (dev, max_pages, _arg(page_table, dev, i32, (self.B, max_pages), "page_table"),
                _arg(sealed_len, dev, i32, (self.B,), "sealed_len"),
                _arg(tail_len, dev, i32, (self.B,), "tail_len"))

    def seal(self, page_table, sealed_len, tail_len, keep_rows=0, stream=None):
        """Seal (tail_len - keep_rows) // 64 blocks of every sequence on every layer and move
        the tail rows that stay to the front; the lengths are left to seal_advance."""
        dev, max_pages, table, sealed, tail = self._lengths(page_table, sealed_len, tail_len)
        st = lib().rapid_kv_seal(*self._ptrs, self.layers, self.dtype, self.B, self.Hkv, self.d,
                                 self.cap, keep_rows, self.n_pages, table, max_pages, sealed, tail,
                                 _raw_stream(stream, dev))
        _check(st, "rapid_kv_seal")

    def seal_advance(self, page_table, sealed_len, tail_len, keep_rows=0, stream=None):
        """sealed_len += 64 n_b, tail_len -= 64 n_b (device, in place)."""
        dev, max_pages, table, sealed, tail = self._lengths(page_table, sealed_len, tail_len)
        st = lib().rapid_kv_seal_advance(sealed, tail, table, self.B, max_pages, self.n_pages,
                                         self.cap, keep_rows, _raw_stream(stream, dev))
        _check(st, "rapid_kv_seal_advance")


def rapid_kv_seal(table, page_table, sealed_len, tail_len, keep_rows=0, stream=None):
    """Q8LayerTable.seal under the C call's name."""
    table.seal(page_table, sealed_len, tail_len, keep_rows, stream)


def rapid_kv_seal_advance(table, page_table, sealed_len, tail_len, keep_rows=0, stream=None):
    """Q8LayerTable.seal_advance under the C call's name."""
    table.seal_advance(page_table, sealed_len, tail_len, keep_rows, stream)


def rapid_verify_attn_q8_workspace_size(B, Hq, Hkv, d, n_q, tail_capacity, max_pages, dtype) -> int:
    return int(lib().rapid_verify_attn_q8_workspace_size(B, Hq, Hkv, d, n_q, tail_capacity,
                                                         max_pages, dtype))


def rapid_verify_attn_q8(Q, K_tail, V_tail, pages, scales, page_table, sealed_len, tail_len,
                         spec_mask, softmax_scale, O, LSE, workspace, stream=None):
    """Verify attention over sealed 8-bit pages, tail rows and the speculative rows."""
    dev = _device_of(Q, "Q")
    if Q.dim() != 4 or K_tail.dim() != 4 or pages.dim() != 5 or page_table.dim() != 2:
        raise RapidError("Q and the tails have 4 dimensions, pages 5, page_table 2")
    B, Hq, n_q, d = shape = Q.shape
    _, Hkv, cap, _ = K_tail.shape
    n_pages, max_pages = pages.shape[0], page_table.shape[1]
    dt, i32 = Q.dtype, torch.int32
    tail_shape = (B, Hkv, cap, d)
    mask_dt = torch.bool if spec_mask is not None and spec_mask.dtype == torch.bool else torch.uint8
    st = lib().rapid_verify_attn_q8(
        _arg(Q, dev, dt, shape, "Q"), _arg(K_tail, dev, dt, tail_shape, "K_tail"),
        _arg(V_tail, dev, dt, tail_shape, "V_tail"),
        _arg(pages, dev, torch.float8_e4m3fn, (n_pages, Hkv, 2, RAPID_Q8_PAGE_TOKENS, d), "pages"),
        _arg(scales, dev, torch.float32, (n_pages, Hkv, 2), "scales"),
        _arg(page_table, dev, i32, (B, max_pages), "page_table"), _dtype_code(Q), B, Hq, Hkv, d,
        n_q, cap, n_pages, max_pages, _arg(sealed_len, dev, i32, (B,), "sealed_len"),
        _arg(tail_len, dev, i32, (B,), "tail_len"),
        _arg(spec_mask, dev, mask_dt, (B, n_q, n_q), "spec_mask"), softmax_scale,
        _arg(O, dev, dt, shape, "O"), _arg(LSE, dev, torch.float32, (B, Hq, n_q), "LSE"),
        _arg(workspace, dev, torch.uint8, (workspace.numel(),), "workspace"), workspace.numel(),
        _raw_stream(stream, dev))
    _check(st, "rapid_verify_attn_q8")


def rapid_device_error(clear: bool = True) -> int:
    return int(lib().rapid_device_error(1 if clear else 0))


def rapid_device_error_info(clear: bool = True):
    words = (ctypes.c_uint32 * 8)()
    if lib().rapid_device_error_info(ctypes.cast(words, ctypes.c_void_p), 1 if clear else 0) != 0:
        raise RapidError("could not read the device error record")
    return list(words)


def rapid_stream_status(stream=None, clear: bool = True) -> int:
    """Synchronise the stream and return RAPID_OK, RAPID_ETIMEOUT (a bounded wait
    inside a kernel gave up), RAPID_EINVAL (a bad device-side input) or RAPID_ECUDA."""
    return int(lib().rapid_stream_status(_stream(stream), 1 if clear else 0))


def rapid_wait_selftest(limit_ns: int, stream=None):
    """Launch the bounded-wait self-test kernel (its wait gives up after limit_ns)."""
    _check(lib().rapid_wait_selftest(int(limit_ns), _stream(stream)), "rapid_wait_selftest")


def rapid_version() -> int:
    return int(lib().rapid_version())


# ---------------------------------------------------------------------------
# Convenience wrappers that allocate outputs and workspaces with torch
# ---------------------------------------------------------------------------

def verify_attn(Q, K, V, prefix_len, spec_mask=None, softmax_scale=0.0, out=None, lse=None,
                workspace=None, stream=None):
    """O [B,Hq,n_q,d] (dtype of Q) and LSE [B,Hq,n_q] float32."""
    B, Hq, n_q, d = Q.shape
    Hkv, cap = K.shape[1], K.shape[2]
    if out is None:
        out = torch.empty_like(Q)
    if lse is None:
        lse = torch.empty((B, Hq, n_q), dtype=torch.float32, device=Q.device)
    if workspace is None:
        nbytes = rapid_verify_attn_workspace_size(B, Hq, Hkv, d, n_q, cap, _dtype_code(Q))
        if nbytes == 0:
            raise RapidError("unsupported verify_attn shape")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=Q.device)
    rapid_verify_attn(Q, K, V, prefix_len, spec_mask, softmax_scale, out, lse, workspace, stream)
    return out, lse


def accept(z, q, tokens, parent=None, T=1.0, eta=1.0, seed=0, tail_clamp=True, want_path=True,
           want_diag=True, workspace=None, stream=None, n_nodes=None):
    """Dict of device tensors n_accepted [B], next_token [B], path [B,n_q], diag [B,n_q,5].

    seed: the Philox key as an int, or a one-element int64 CUDA tensor that the kernels read
    when they run.  n_nodes: None, or int32 [B] node counts of drafts shorter than n_q.
    Either one goes through rapid_accept_ex."""
    B, n_q, V = z.shape
    dev = z.device
    n_acc = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    path = torch.empty((B, n_q), dtype=torch.int32, device=dev) if want_path else None
    diag = torch.empty((B, n_q, 5), dtype=torch.float32, device=dev) if want_diag else None
    if workspace is None:
        nbytes = rapid_accept_workspace_size(B, n_q, V)
        if nbytes == 0:
            raise RapidError("unsupported accept shape")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    flags = RAPID_ACCEPT_TAIL_CLAMP if tail_clamp else 0
    if isinstance(seed, torch.Tensor) or n_nodes is not None:
        rapid_accept_ex(z, q, tokens, parent, n_nodes, T, eta, seed, flags, n_acc, nxt, path,
                        diag, workspace, stream)
    else:
        rapid_accept(z, q, tokens, parent, T, eta, seed, flags, n_acc, nxt, path, diag,
                     workspace, stream)
    return dict(n_accepted=n_acc, next_token=nxt, path=path, diag=diag)


def lm_head_accept(hidden, W_lm, q, tokens, parent=None, T=1.0, eta=1.0, seed=0, tail_clamp=True,
                   want_path=True, want_diag=True, workspace=None, stream=None):
    """accept() on the logits of the verify rows' hidden states [B*n_q, hidden_dim]."""
    B, n_q, V = q.shape
    dev = q.device
    n_acc = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    path = torch.empty((B, n_q), dtype=torch.int32, device=dev) if want_path else None
    diag = torch.empty((B, n_q, 5), dtype=torch.float32, device=dev) if want_diag else None
    if workspace is None:
        nbytes = rapid_lm_head_accept_workspace_size(B, n_q, V)
        if nbytes == 0:
            raise RapidError("unsupported lm_head_accept shape")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    flags = RAPID_ACCEPT_TAIL_CLAMP if tail_clamp else 0
    rapid_lm_head_accept(hidden, W_lm, q, tokens, parent, T, eta, seed, flags, n_acc, nxt, path,
                         diag, workspace, stream)
    return dict(n_accepted=n_acc, next_token=nxt, path=path, diag=diag)


def _on(stream):
    """What a wrapper allocates belongs to the stream that its kernels run on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def qkv_append(q, k, v, K, V, prefix_len, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
               interleaved=False, pos_offset=None, row_offset=None, n_rows=None, out=None,
               stream=None):
    """Queries [B, Hq, n, d] of the projection rows q [B, n, Hq, d], k and v [B, n, Hkv, d], with
    norm (where a weight is given) and rotation (where inv_freq is given); keys and values go to
    rows prefix_len[b] + i of K and V [B, Hkv, capacity, d].

    Where n_rows cuts a sequence short, its rows of `out` behind the count are left as they are
    (unset memory in an `out` made here)."""
    if out is None:
        B, n, Hq, d = q.shape
        with _on(stream):
            out = torch.empty((B, Hq, n, d), dtype=q.dtype, device=q.device)
    rapid_qkv_append(q, k, v, q_weight, k_weight, eps, inv_freq,
                     RAPID_ROPE_INTERLEAVED if interleaved else 0, prefix_len, pos_offset,
                     row_offset, n_rows, out, K, V, stream)
    return out


@functools.lru_cache(maxsize=256)
def _attn_q8_bytes(device, *sizes):
    nbytes = rapid_verify_attn_q8_workspace_size(*sizes)
    if nbytes == 0:
        raise RapidError("unsupported verify_attn_q8 shape")
    return nbytes


_held = threading.local()


def _scratch(dev, nbytes):
    """Scratch for one call on the current stream.  It is kept for the next call that the same
    host thread makes on the same stream, which the stream orders behind this one, until the
    thread ends; a call that is being captured gets memory of its own, because its graph may run
    on any stream.  A stream is known by its handle, as in torch's allocator: one that was made
    outside torch may be destroyed only after its work is done."""
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
    key = (dev, torch._C._cuda_getCurrentRawStream(dev))
    held = _held.__dict__
    t = held.get(key)
    if t is None or t.numel() < nbytes:
        t = held[key] = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{dev}")
    return t


def verify_attn_q8(Q, K_tail, V_tail, pages, scales, page_table, sealed_len, tail_len,
                   spec_mask=None, softmax_scale=0.0, out=None, lse=None, workspace=None,
                   stream=None):
    """O [B,Hq,n_q,d] (dtype of Q) and LSE [B,Hq,n_q] float32 over an 8-bit history.

    Without a workspace the call uses scratch that the host thread keeps for each stream (a few
    megabytes); do not destroy a stream made outside torch while its calls are pending.  Calls
    that may overlap in other ways (two graphs of one memory pool) need workspaces of their own."""
    if stream is not None:
        with torch.cuda.stream(stream):    # what is allocated here belongs to that stream
            return verify_attn_q8(Q, K_tail, V_tail, pages, scales, page_table, sealed_len,
                                  tail_len, spec_mask, softmax_scale, out, lse, workspace)
    B, Hq, n_q, d = Q.shape
    dev = Q.device
    if out is None:
        out = torch.empty_like(Q)
    if lse is None:
        lse = torch.empty((B, Hq, n_q), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _scratch(_device_of(Q, "Q"), _attn_q8_bytes(
            dev.index, B, Hq, K_tail.shape[1], d, n_q, K_tail.shape[2], page_table.shape[1],
            _dtype_code(Q)))
    rapid_verify_attn_q8(Q, K_tail, V_tail, pages, scales, page_table, sealed_len, tail_len,
                         spec_mask, softmax_scale, out, lse, workspace)
    return out, lse
