"""ctypes binding of libdsa.so (include/dsa.h).  Argument marshalling only.

Every function keeps the C name.  Tensors are torch tensors on the GPU (their data pointers
are passed through); the stream defaults to torch's current stream.  A non-OK status raises
DsaError carrying the library's message.  There is no fallback: if the shared library is
missing the first call raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_LAYER_SHARED = 0
DSA_LAYER_FULL = 1
DSA_IDX_ROPE_Q = 1 << 0
DSA_IDX_ROPE_K = 1 << 1
DSA_IDX_INDEPENDENT_ROWS = 1 << 2
DSA_ROPE_SCALE_NONE, DSA_ROPE_SCALE_LINEAR, DSA_ROPE_SCALE_YARN = 0, 1, 2
DSA_BF16, DSA_F32 = 0, 1
DSA_ROPE_INTERLEAVED = 1 << 0
DSA_ROPE_INVERSE = 1 << 1
DSA_CACHE_BF16, DSA_CACHE_FP8 = 0, 1
DSA_CACHE_ROPE = 1 << 8

STATUS_NAMES = {0: "DSA_OK", 1: "DSA_ERR_ARG", 2: "DSA_ERR_SHAPE", 3: "DSA_ERR_NO_DONOR", 4: "DSA_ERR_UNSUPPORTED",
                5: "DSA_ERR_CUDA", 6: "DSA_ERR_WORKSPACE", 7: "DSA_ERR_TIMEOUT", 8: "DSA_ERR_DEVICE"}
EXPORTED = ("dsa_status_string", "dsa_last_error", "dsa_donor_table", "dsa_rope_table", "dsa_indexer_workspace_size",
            "dsa_indexer_topk", "dsa_sparse_attn_workspace_size", "dsa_sparse_attn", "dsa_index_cache_create",
            "dsa_index_cache_donor", "dsa_index_cache_indices", "dsa_index_cache_destroy",
            "dsa_layers_workspace_size", "indexshare_layers_forward", "dsa_workspace_status",
            "dsa_indexer_topk_static", "dsa_profile_enable", "dsa_profile_indexer_last", "dsa_mtp_indexshare_step",
            "dsa_indexer_topk_paged", "dsa_sparse_attn_paged", "dsa_indexer_projections", "dsa_sparse_attn_backward",
            "dsa_indexer_static_status", "dsa_profile_read", "dsa_debug_pipeline",
            "dsa_indexer_backward_workspace_size", "dsa_indexer_backward",
            "dsa_sparse_attn_backward_workspace_size", "dsa_rope_table_scaled", "dsa_rope_apply",
            "dsa_latent_cache_write", "dsa_latent_cache_read", "dsa_latent_attn_workspace_size",
            "dsa_latent_attn_paged", "dsa_mtp_verify", "dsa_latent_attn_shared_workspace_size",
            "dsa_latent_attn_shared", "dsa_latent_key_weights_workspace_size", "dsa_latent_key_weights",
            "dsa_latent_cache_evict_workspace_size", "dsa_latent_cache_evict")

PROFILE_KINDS = {0: "rope", 1: "ranges", 2: "indexer", 3: "select", 4: "attn_prep", 5: "attn", 6: "attn_bwd",
                 7: "proj", 8: "indexer_bwd", 9: "cache", 10: "verify"}


class DsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))
        super().__init__(f"{self.name}: {message}")


class IndexerDesc(C.Structure):
    _fields_ = [("n_q", C.c_int32), ("n_kv", C.c_int32), ("n_heads", C.c_int32), ("head_dim", C.c_int32),
                ("rope_dim", C.c_int32), ("topk", C.c_int32), ("max_len", C.c_int32), ("flags", C.c_uint32)]


class AttnDesc(C.Structure):
    _fields_ = [("n_q", C.c_int32), ("n_kv", C.c_int32), ("n_heads", C.c_int32), ("d_qk", C.c_int32),
                ("d_v", C.c_int32), ("topk", C.c_int32), ("softmax_scale", C.c_float), ("flags", C.c_uint32)]


class ProfileRecord(C.Structure):
    _fields_ = [("kind", C.c_int32), ("ms", C.c_float)]


class LayerIO(C.Structure):
    _fields_ = [("q_idx", C.c_void_p), ("k_idx", C.c_void_p), ("w", C.c_void_p), ("q", C.c_void_p),
                ("kv", C.c_void_p), ("out", C.c_void_p), ("lse", C.c_void_p)]


class RopeScaling(C.Structure):
    """dsa_rope_scaling: a scaled RoPE table (see rope_scaling_linear and rope_scaling_yarn)."""
    _fields_ = [("kind", C.c_int32), ("orig_len", C.c_int32), ("factor", C.c_double), ("beta_fast", C.c_double),
                ("beta_slow", C.c_double), ("mscale", C.c_double)]


class RopeDesc(C.Structure):
    _fields_ = [("n_tokens", C.c_int32), ("n_heads", C.c_int32), ("rope_dim", C.c_int32), ("dtype", C.c_int32),
                ("x_token_stride", C.c_int64), ("x_head_stride", C.c_int64), ("out_token_stride", C.c_int64),
                ("out_head_stride", C.c_int64), ("flags", C.c_uint32)]


class LatentCache(C.Structure):
    """dsa_latent_cache (see latent_cache)."""
    _fields_ = [("latent", C.c_void_p), ("scale", C.c_void_p), ("rope", C.c_void_p), ("n_rows", C.c_int32),
                ("format", C.c_int32)]
    device = None       # ordinal of the tensors' device, where latent_cache made it


class CacheWriteDesc(C.Structure):
    _fields_ = [("n_tokens", C.c_int32), ("flags", C.c_uint32), ("kv_stride", C.c_int64)]


class SharedRows(C.Structure):
    """dsa_shared_rows (see shared_rows)."""
    _fields_ = [("group_start", C.c_void_p), ("prefix_len", C.c_void_p), ("n_groups", C.c_int32),
                ("max_rows", C.c_int32)]
    device = None       # ordinal of the tensors' device, where shared_rows made it


class EvictDesc(C.Structure):
    _fields_ = [("n_seq", C.c_int32), ("n_keep", C.c_int32), ("n_first", C.c_int32), ("n_last", C.c_int32)]


class VerifyDesc(C.Structure):
    _fields_ = [("n_seq", C.c_int32), ("n_draft", C.c_int32), ("vocab", C.c_int32), ("dtype", C.c_int32),
                ("target_stride", C.c_int64), ("draft_stride", C.c_int64)]


_lib: Optional[C.CDLL] = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run dsa_indexer_cross_gb300.build.build() first")
        L = C.CDLL(LIB_PATH)
        st, vp, i32, u32, sz = C.c_int, C.c_void_p, C.c_int32, C.c_uint32, C.c_size_t
        P = C.POINTER
        L.dsa_status_string.restype = C.c_char_p
        L.dsa_status_string.argtypes = [st]
        L.dsa_last_error.restype = C.c_char_p
        L.dsa_last_error.argtypes = []
        L.dsa_donor_table.restype = st
        L.dsa_donor_table.argtypes = [i32, P(C.c_uint8), P(i32)]
        L.dsa_rope_table.restype = st
        L.dsa_rope_table.argtypes = [C.c_double, i32, i32, P(C.c_float)]
        L.dsa_indexer_workspace_size.restype = st
        L.dsa_indexer_workspace_size.argtypes = [P(IndexerDesc), P(sz)]
        L.dsa_indexer_topk.restype = st
        L.dsa_indexer_topk.argtypes = [P(IndexerDesc), vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        L.dsa_sparse_attn_workspace_size.restype = st
        L.dsa_sparse_attn_workspace_size.argtypes = [P(AttnDesc), P(sz)]
        L.dsa_sparse_attn.restype = st
        L.dsa_sparse_attn.argtypes = [P(AttnDesc), vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dsa_index_cache_create.restype = st
        L.dsa_index_cache_create.argtypes = [i32, P(C.c_uint8), i32, i32, P(vp), P(vp)]
        L.dsa_index_cache_donor.restype = st
        L.dsa_index_cache_donor.argtypes = [vp, i32, P(i32)]
        L.dsa_index_cache_indices.restype = vp
        L.dsa_index_cache_indices.argtypes = [vp, i32]
        L.dsa_index_cache_destroy.restype = None
        L.dsa_index_cache_destroy.argtypes = [vp]
        L.dsa_layers_workspace_size.restype = st
        L.dsa_layers_workspace_size.argtypes = [P(IndexerDesc), P(AttnDesc), P(sz)]
        L.indexshare_layers_forward.restype = st
        L.indexshare_layers_forward.argtypes = [P(IndexerDesc), P(AttnDesc), i32, P(C.c_uint8), P(LayerIO), vp, vp,
                                                vp, vp, vp, i32, vp, vp, sz, vp]
        L.dsa_workspace_status.restype = st
        L.dsa_workspace_status.argtypes = [vp, vp, P(u32)]
        L.dsa_profile_enable.restype = st
        L.dsa_profile_enable.argtypes = [i32]
        L.dsa_profile_indexer_last.restype = st
        L.dsa_profile_indexer_last.argtypes = [P(C.c_float), i32]
        L.dsa_indexer_topk_static.restype = st
        L.dsa_indexer_topk_static.argtypes = [P(IndexerDesc), vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
        L.dsa_indexer_static_status.restype = st
        L.dsa_indexer_static_status.argtypes = [vp, P(u32)]
        L.dsa_debug_pipeline.restype = st
        L.dsa_debug_pipeline.argtypes = [i32, C.c_uint64]
        L.dsa_profile_read.restype = st
        L.dsa_profile_read.argtypes = [P(ProfileRecord), i32, P(i32)]
        L.dsa_sparse_attn_backward.restype = st
        L.dsa_sparse_attn_backward_workspace_size.restype = st
        L.dsa_sparse_attn_backward_workspace_size.argtypes = [P(AttnDesc), P(sz)]
        L.dsa_sparse_attn_backward.argtypes = [P(AttnDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dsa_indexer_backward_workspace_size.restype = st
        L.dsa_indexer_backward_workspace_size.argtypes = [P(IndexerDesc), P(sz)]
        L.dsa_indexer_backward.restype = st
        L.dsa_indexer_backward.argtypes = [P(IndexerDesc), vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                           sz, vp]
        L.dsa_indexer_projections.restype = st
        L.dsa_indexer_projections.argtypes = [P(ProjDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dsa_indexer_topk_paged.restype = st
        L.dsa_indexer_topk_paged.argtypes = [P(IndexerDesc), vp, vp, vp, vp, P(PagedCache), vp, i32, vp, vp, vp, sz, vp]
        L.dsa_sparse_attn_paged.restype = st
        L.dsa_sparse_attn_paged.argtypes = [P(AttnDesc), vp, vp, vp, P(PagedCache), vp, vp, vp, sz, vp]
        L.dsa_mtp_indexshare_step.restype = st
        L.dsa_mtp_indexshare_step.argtypes = [P(IndexerDesc), P(AttnDesc), i32, P(LayerIO), vp, vp, vp, vp, vp, i32,
                                              vp, vp, sz, vp]
        L.dsa_rope_table_scaled.restype = st
        L.dsa_rope_table_scaled.argtypes = [C.c_double, i32, i32, P(RopeScaling), P(C.c_float)]
        L.dsa_rope_apply.restype = st
        L.dsa_rope_apply.argtypes = [P(RopeDesc), vp, vp, vp, i32, vp, vp, sz, vp]
        L.dsa_latent_cache_write.restype = st
        L.dsa_latent_cache_write.argtypes = [P(CacheWriteDesc), vp, vp, vp, vp, i32, P(LatentCache), vp, sz, vp]
        L.dsa_latent_cache_read.restype = st
        L.dsa_latent_cache_read.argtypes = [P(LatentCache), P(PagedCache), i32, vp, vp, i32, vp, sz, vp]
        L.dsa_latent_attn_workspace_size.restype = st
        L.dsa_latent_attn_workspace_size.argtypes = [P(AttnDesc), P(sz)]
        L.dsa_latent_attn_paged.restype = st
        L.dsa_latent_attn_paged.argtypes = [P(AttnDesc), vp, P(LatentCache), vp, P(PagedCache), vp, vp, vp, sz, vp]
        L.dsa_latent_attn_shared_workspace_size.restype = st
        L.dsa_latent_attn_shared_workspace_size.argtypes = [P(AttnDesc), P(SharedRows), P(sz)]
        L.dsa_latent_attn_shared.restype = st
        L.dsa_latent_attn_shared.argtypes = [P(AttnDesc), vp, P(LatentCache), P(SharedRows), P(PagedCache), vp, vp, vp, sz,
                                             vp]
        L.dsa_latent_key_weights_workspace_size.restype = st
        L.dsa_latent_key_weights_workspace_size.argtypes = [P(AttnDesc), P(PagedCache), P(sz)]
        L.dsa_latent_key_weights.restype = st
        L.dsa_latent_key_weights.argtypes = [P(AttnDesc), vp, P(LatentCache), P(PagedCache), vp, vp, vp, C.c_int64, vp, sz,
                                             vp]
        L.dsa_latent_cache_evict_workspace_size.restype = st
        L.dsa_latent_cache_evict_workspace_size.argtypes = [P(EvictDesc), P(sz)]
        L.dsa_latent_cache_evict.restype = st
        L.dsa_latent_cache_evict.argtypes = [P(EvictDesc), P(LatentCache), P(PagedCache), vp, C.c_int64, P(LatentCache),
                                             P(PagedCache), vp, vp, C.c_int64, vp, vp, sz, vp]
        L.dsa_mtp_verify.restype = st
        L.dsa_mtp_verify.argtypes = [P(VerifyDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != 0:
        raise DsaError(status, lib().dsa_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Device address of a contiguous CUDA tensor (every tensor argument of libdsa's GPU calls is
    device memory; a host tensor is refused here rather than handed to a kernel)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libdsa must be CUDA tensors (device memory)")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdsa must be contiguous")
    return t.data_ptr()


def _want(t: torch.Tensor, dtype, numel: int, name: str) -> None:
    """Refuse a tensor of the wrong type or too few elements before its address reaches a kernel
    (the C ABI takes bare pointers and cannot check either)."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")


# (None in a torch without CUDA, whose calls never get here)
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:      # the handle alone: a Stream object costs as much as a small launch
        return _raw_stream(_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace for one call, out of the memory of the stream that runs it: the allocator hands memory on
    in the order of one stream's work, so another stream's block may be written, or given away, while this call
    is still to use it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _arg(t: torch.Tensor, dtype, numel: int, name: str, dev: int) -> int:
    """_want and _ptr in one, on device `dev`, for the calls of a few microseconds."""
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= numel and t.is_contiguous():
        return t.data_ptr()
    _want(t, dtype, numel, name)
    _ptr(t)
    raise ValueError(f"{name} is on {t.device}, but the call's other tensors are on cuda:{dev}")


def _current_device(t: torch.Tensor, name: str, *handles) -> int:
    """The current device, which holds `t` and the tensors of the cache and page-table handles."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: tensors passed to libdsa must be CUDA tensors (device memory)")
    if dev != _device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_device()}")
    for h in handles:
        if h.device is not None and h.device != dev:
            raise ValueError(f"{name} is on {t.device}, but the {type(h).__name__}'s tensors are on cuda:{h.device}")
    return dev


def _one_device(*tensors) -> int:
    """The ordinal of the device that holds every tensor of a handle."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"a handle's tensors must be on one device, not {tensors[0].device} and {t.device}")
    return dev


def _u8(types: Sequence[int]):
    return (C.c_uint8 * len(types))(*[int(x) for x in types])


def types_to_u8(indexer_types: Sequence) -> list:
    """'full'/'shared' strings (as in a released config) or 0/1 ints -> 0/1 ints."""
    out = []
    for t in indexer_types:
        if isinstance(t, str):
            out.append(DSA_LAYER_FULL if t == "full" else DSA_LAYER_SHARED if t == "shared" else 255)
        else:
            out.append(int(t))
    return out


# ------------------------------------------------------------------------------ schedule

def dsa_donor_table(indexer_types: Sequence) -> list:
    types = types_to_u8(indexer_types)
    donors = (C.c_int32 * max(1, len(types)))()
    _check(lib().dsa_donor_table(len(types), _u8(types), donors))
    return list(donors)[:len(types)]


def dsa_rope_table(theta: float, rope_dim: int, n_pos: int) -> torch.Tensor:
    """Host float32 tensor [n_pos, rope_dim/2, 2] of (cos, sin)."""
    out = torch.empty((n_pos, max(rope_dim // 2, 1), 2), dtype=torch.float32)
    _check(lib().dsa_rope_table(float(theta), int(rope_dim), int(n_pos),
                                C.cast(out.data_ptr(), C.POINTER(C.c_float))))
    return out


# ------------------------------------------------------------------------------ indexer

def indexer_desc(n_q, n_kv, n_heads, head_dim, rope_dim, topk, max_len, flags) -> IndexerDesc:
    return IndexerDesc(n_q, n_kv, n_heads, head_dim, rope_dim, topk, max_len, flags)


def dsa_indexer_workspace_size(desc: IndexerDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_indexer_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def _indexer_args(desc: IndexerDesc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx_out, score_out) -> None:
    n_q, n_kv, H, d, k = desc.n_q, desc.n_kv, desc.n_heads, desc.head_dim, desc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, dt, n, name in ((q_idx, bf, n_q * H * d, "q_idx"), (k_idx, bf, n_kv * d, "k_idx"), (w, f32, n_q * H, "w"),
                           (q_pos, i32, n_q, "q_pos"), (k_pos, i32, n_kv, "k_pos"), (ks, i32, n_q, "ks"),
                           (ke, i32, n_q, "ke"), (rope_cs, f32, 0, "rope_cs"), (idx_out, i32, n_q * k, "idx_out"),
                           (score_out, f32, n_q * k, "score_out")):
        if t is not None:
            _want(t, dt, n, name)


def dsa_indexer_topk(desc: IndexerDesc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx_out, score_out=None,
                     ws=None, stream=None) -> torch.Tensor:
    _indexer_args(desc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx_out, score_out)
    if ws is None:
        ws = _workspace(dsa_indexer_workspace_size(desc), idx_out.device, stream)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().dsa_indexer_topk(C.byref(desc), _ptr(q_idx), _ptr(k_idx), _ptr(w), _ptr(q_pos), _ptr(k_pos),
                                  _ptr(ks), _ptr(ke), _ptr(rope_cs), n_pos, _ptr(idx_out), _ptr(score_out),
                                  _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def dsa_indexer_topk_static(desc: IndexerDesc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx_out,
                            score_out=None, stream=None) -> None:
    """dsa_indexer_topk with the library's static device scratch instead of a workspace."""
    _indexer_args(desc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx_out, score_out)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().dsa_indexer_topk_static(C.byref(desc), _ptr(q_idx), _ptr(k_idx), _ptr(w), _ptr(q_pos), _ptr(k_pos),
                                         _ptr(ks), _ptr(ke), _ptr(rope_cs), n_pos, _ptr(idx_out), _ptr(score_out),
                                         _stream(stream)))


def dsa_indexer_backward_workspace_size(desc: IndexerDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_indexer_backward_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def dsa_indexer_backward(desc: IndexerDesc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx, d_score, dq_idx,
                         dk_idx, dw, ws=None, stream=None) -> torch.Tensor:
    """Gradients of the selected scores: dq_idx (written), dk_idx and dw (zeroed, then
    accumulated), fp32, for the upstream d_score aligned with the forward's idx."""
    _indexer_args(desc, q_idx, k_idx, w, q_pos, k_pos, ks, ke, rope_cs, idx, None)
    n_q, n_kv, H, d, k = desc.n_q, desc.n_kv, desc.n_heads, desc.head_dim, desc.topk
    f32 = torch.float32
    for t, n, name in ((d_score, n_q * k, "d_score"), (dq_idx, n_q * H * d, "dq_idx"), (dk_idx, n_kv * d, "dk_idx"),
                       (dw, n_q * H, "dw")):
        _want(t, f32, n, name)
    if ws is None:
        ws = _workspace(dsa_indexer_backward_workspace_size(desc), dq_idx.device, stream)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().dsa_indexer_backward(C.byref(desc), _ptr(q_idx), _ptr(k_idx), _ptr(w), _ptr(q_pos), _ptr(k_pos),
                                      _ptr(ks), _ptr(ke), _ptr(rope_cs), n_pos, _ptr(idx), _ptr(d_score),
                                      _ptr(dq_idx), _ptr(dk_idx), _ptr(dw), _ptr(ws), ws.numel(), _stream(stream)))
    return ws


# ------------------------------------------------------------------------------ attention

def attn_desc(n_q, n_kv, n_heads, topk, softmax_scale, d_qk=576, d_v=512) -> AttnDesc:
    return AttnDesc(n_q, n_kv, n_heads, d_qk, d_v, topk, softmax_scale, 0)


def dsa_sparse_attn_workspace_size(desc: AttnDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_sparse_attn_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def dsa_sparse_attn(desc: AttnDesc, q, kv, idx, ks, out, lse=None, ws=None, stream=None) -> torch.Tensor:
    n_q, n_kv, H, k = desc.n_q, desc.n_kv, desc.n_heads, desc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, dt, n, name in ((q, bf, n_q * H * desc.d_qk, "q"), (kv, bf, n_kv * desc.d_qk, "kv"), (idx, i32, n_q * k, "idx"),
                           (ks, i32, n_q, "ks"), (out, bf, n_q * H * desc.d_v, "out"), (lse, f32, n_q * H, "lse")):
        if t is not None:
            _want(t, dt, n, name)
    if ws is None:
        ws = _workspace(dsa_sparse_attn_workspace_size(desc), out.device, stream)
    _check(lib().dsa_sparse_attn(C.byref(desc), _ptr(q), _ptr(kv), _ptr(idx), _ptr(ks), _ptr(out), _ptr(lse),
                                 _ptr(ws), ws.numel(), _stream(stream)))
    return ws


# ------------------------------------------------------------------------------ index cache

class IndexCache:
    """Owns a dsa_index_cache handle and the per-full-layer device index buffers."""

    def __init__(self, indexer_types: Sequence, n_q: int, topk: int, device="cuda"):
        self.types = types_to_u8(indexer_types)
        self.n_q, self.topk = n_q, topk
        self.buffers = [torch.full((n_q, topk), -1, dtype=torch.int32, device=device)
                        if t == DSA_LAYER_FULL else None for t in self.types]
        ptrs = (C.c_void_p * len(self.types))(*[b.data_ptr() if b is not None else None for b in self.buffers])
        h = C.c_void_p()
        _check(lib().dsa_index_cache_create(len(self.types), _u8(self.types), n_q, topk, ptrs, C.byref(h)))
        self.handle = h

    def donor(self, layer: int) -> int:
        d = C.c_int32(0)
        _check(lib().dsa_index_cache_donor(self.handle, layer, C.byref(d)))
        return d.value

    def indices_ptr(self, layer: int) -> int:
        p = lib().dsa_index_cache_indices(self.handle, layer)
        if not p:
            raise DsaError(1, lib().dsa_last_error().decode())
        return p

    def indices(self, layer: int) -> torch.Tensor:
        return self.buffers[self.donor(layer)]

    def close(self):
        if getattr(self, "handle", None):
            lib().dsa_index_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------------------ layer loop

def dsa_layers_workspace_size(idesc: IndexerDesc, adesc: AttnDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_layers_workspace_size(C.byref(idesc), C.byref(adesc), C.byref(n)))
    return n.value


def indexshare_layers_forward(idesc: IndexerDesc, adesc: AttnDesc, indexer_types: Sequence, layers: Sequence[dict],
                              ks, ke, q_pos, k_pos, rope_cs, cache: IndexCache, ws=None, stream=None):
    """layers[l]: dict with 'q', 'kv', 'out' (+ 'lse') and, on full layers, 'q_idx', 'k_idx', 'w'."""
    types = types_to_u8(indexer_types)
    io = (LayerIO * len(layers))()
    for l, L in enumerate(layers):
        io[l] = LayerIO(_ptr(L.get("q_idx")), _ptr(L.get("k_idx")), _ptr(L.get("w")), _ptr(L["q"]), _ptr(L["kv"]),
                        _ptr(L["out"]), _ptr(L.get("lse")))
    if ws is None:
        ws = _workspace(dsa_layers_workspace_size(idesc, adesc), layers[0]["q"].device, stream)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().indexshare_layers_forward(C.byref(idesc), C.byref(adesc), len(types), _u8(types), io, _ptr(ks),
                                           _ptr(ke), _ptr(q_pos), _ptr(k_pos), _ptr(rope_cs), n_pos, cache.handle,
                                           _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def dsa_sparse_attn_backward_workspace_size(desc: AttnDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_sparse_attn_backward_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def dsa_sparse_attn_backward(desc: AttnDesc, q, kv, idx, ks, out, lse, d_out, dq, dkv, ws=None, stream=None):
    """dq (written) and dkv (zeroed, then accumulated), fp32, for the upstream gradient d_out."""
    n_q, n_kv, H, k = desc.n_q, desc.n_kv, desc.n_heads, desc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, dt, n, name in ((q, bf, n_q * H * desc.d_qk, "q"), (kv, bf, n_kv * desc.d_qk, "kv"), (idx, i32, n_q * k, "idx"),
                           (ks, i32, n_q, "ks"), (out, bf, n_q * H * desc.d_v, "out"), (lse, f32, n_q * H, "lse"),
                           (d_out, bf, n_q * H * desc.d_v, "d_out"), (dq, f32, n_q * H * desc.d_qk, "dq"),
                           (dkv, f32, n_kv * desc.d_qk, "dkv")):
        _want(t, dt, n, name)
    if ws is None:
        ws = _workspace(dsa_sparse_attn_backward_workspace_size(desc), q.device, stream)
    _check(lib().dsa_sparse_attn_backward(C.byref(desc), _ptr(q), _ptr(kv), _ptr(idx), _ptr(ks), _ptr(out), _ptr(lse),
                                          _ptr(d_out), _ptr(dq), _ptr(dkv), _ptr(ws), ws.numel(), _stream(stream)))
    return ws


class ProjDesc(C.Structure):
    _fields_ = [("n_tokens", C.c_int32), ("d_hidden", C.c_int32), ("d_q", C.c_int32), ("n_heads", C.c_int32),
                ("head_dim", C.c_int32), ("ln_eps", C.c_float)]


def dsa_indexer_projections(desc: "ProjDesc", x, q_latent, wq_b, wk, k_norm_w, k_norm_b, weights_proj, q_idx, k_idx,
                            w, ws=None, stream=None):
    """q_idx = q_latent wq_b^T, k_idx = LayerNorm(x wk^T) (k_norm weight / bias), w = x weights_proj^T."""
    T, dh, dq, H, d = desc.n_tokens, desc.d_hidden, desc.d_q, desc.n_heads, desc.head_dim
    bf, f32 = torch.bfloat16, torch.float32
    for t, dt, n, name in ((x, bf, T * dh, "x"), (q_latent, bf, T * dq, "q_latent"), (wq_b, bf, H * d * dq, "wq_b"),
                           (wk, bf, d * dh, "wk"), (k_norm_w, f32, d, "k_norm_w"), (k_norm_b, f32, d, "k_norm_b"),
                           (weights_proj, bf, H * dh, "weights_proj"), (q_idx, bf, T * H * d, "q_idx"),
                           (k_idx, bf, T * d, "k_idx"), (w, f32, T * H, "w")):
        _want(t, dt, n, name)
    if ws is None:
        ws = _workspace(256, x.device, stream)
    _check(lib().dsa_indexer_projections(C.byref(desc), _ptr(x), _ptr(q_latent), _ptr(wq_b), _ptr(wk), _ptr(k_norm_w),
                                         _ptr(k_norm_b), _ptr(weights_proj), _ptr(q_idx), _ptr(k_idx), _ptr(w),
                                         _ptr(ws), ws.numel(), _stream(stream)))
    return ws


DSA_PAGE_ROWS = 128


class PagedCache(C.Structure):
    """dsa_paged_cache: row t's logical key j sits at cache row
    block_table[t, j // page_rows] * page_rows + j % page_rows, valid for j < seq_len[t]."""
    _fields_ = [("block_table", C.c_void_p), ("seq_len", C.c_void_p), ("max_pages", C.c_int32),
                ("n_pages", C.c_int32), ("page_rows", C.c_int32)]
    rows = device = None       # rows that both tables have, their device's ordinal, where paged_cache made it


def paged_cache(block_table: torch.Tensor, seq_len: torch.Tensor, n_pages: int) -> PagedCache:
    """block_table: int32 [n_q, max_pages] device tensor; seq_len: int32 [n_q] (kept alive by the caller).
    Calls of at most as many rows as the shorter of the two has."""
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [rows, max_pages], got {block_table.dim()} dims")
    _want(block_table, torch.int32, 0, "block_table")
    _want(seq_len, torch.int32, 0, "seq_len")
    pages = PagedCache(_ptr(block_table), _ptr(seq_len), block_table.shape[1], n_pages, DSA_PAGE_ROWS)
    pages.rows = min(block_table.shape[0], seq_len.numel())
    pages.device = _one_device(block_table, seq_len)
    return pages


def _paged_args(pages: PagedCache, rows: int) -> None:
    if pages.rows is not None and rows > pages.rows:
        raise ValueError(f"paged cache: a call of {rows} rows, block_table and seq_len have {pages.rows}")
    if rows and not (pages.block_table and pages.seq_len):      # (an empty tensor has no address)
        raise ValueError("paged cache: block_table and seq_len must be set")


def dsa_indexer_topk_paged(desc: IndexerDesc, q_idx, k_cache, w, q_pos, pages: PagedCache, rope_cs, idx_out,
                           score_out=None, ws=None, stream=None):
    n_q, H, d, k = desc.n_q, desc.n_heads, desc.head_dim, desc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, dt, n, name in ((q_idx, bf, n_q * H * d, "q_idx"), (k_cache, bf, desc.n_kv * d, "k_cache"),
                           (w, f32, n_q * H, "w"), (q_pos, i32, n_q, "q_pos"), (rope_cs, f32, 0, "rope_cs"),
                           (idx_out, i32, n_q * k, "idx_out"), (score_out, f32, n_q * k, "score_out")):
        if t is not None:
            _want(t, dt, n, name)
    _paged_args(pages, n_q)
    if ws is None:
        ws = _workspace(dsa_indexer_workspace_size(desc), q_idx.device, stream)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().dsa_indexer_topk_paged(C.byref(desc), _ptr(q_idx), _ptr(k_cache), _ptr(w), _ptr(q_pos),
                                        C.byref(pages), _ptr(rope_cs), n_pos, _ptr(idx_out), _ptr(score_out),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def dsa_sparse_attn_paged(desc: AttnDesc, q, kv_cache, idx, pages: PagedCache, out, lse=None, ws=None, stream=None):
    n_q, H, k = desc.n_q, desc.n_heads, desc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, dt, n, name in ((q, bf, n_q * H * desc.d_qk, "q"), (kv_cache, bf, desc.n_kv * desc.d_qk, "kv_cache"),
                           (idx, i32, n_q * k, "idx"), (out, bf, n_q * H * desc.d_v, "out"), (lse, f32, n_q * H, "lse")):
        if t is not None:
            _want(t, dt, n, name)
    _paged_args(pages, n_q)
    if ws is None:
        ws = _workspace(dsa_sparse_attn_workspace_size(desc), q.device, stream)
    _check(lib().dsa_sparse_attn_paged(C.byref(desc), _ptr(q), _ptr(kv_cache), _ptr(idx), C.byref(pages), _ptr(out),
                                       _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return ws


# ------------------------------------------------------------------------------ rotary positions

def rope_scaling_linear(factor: float, mscale: float = 1.0) -> RopeScaling:
    """Position interpolation: every frequency divided by factor."""
    return RopeScaling(DSA_ROPE_SCALE_LINEAR, 0, float(factor), 0.0, 0.0, float(mscale))


def rope_scaling_yarn(factor: float, orig_len: int, beta_fast: float = 32.0, beta_slow: float = 1.0,
                      mscale: float = 1.0) -> RopeScaling:
    """YaRN: frequencies that turn often within orig_len kept, slow ones divided by factor."""
    return RopeScaling(DSA_ROPE_SCALE_YARN, int(orig_len), float(factor), float(beta_fast), float(beta_slow),
                       float(mscale))


def dsa_rope_table_scaled(theta: float, rope_dim: int, n_pos: int, scaling: Optional[RopeScaling] = None) -> torch.Tensor:
    """Host float32 tensor [n_pos, rope_dim/2, 2] of (cos, sin), scaled for long contexts."""
    out = torch.empty((max(n_pos, 0), max(rope_dim // 2, 1), 2), dtype=torch.float32)
    _check(lib().dsa_rope_table_scaled(float(theta), int(rope_dim), int(n_pos), C.byref(scaling) if scaling else None,
                                       C.cast(out.data_ptr(), C.POINTER(C.c_float))))
    return out


def _heads_view(t: torch.Tensor, name: str):
    """(token stride, head stride) of a [tokens, heads, rope_dim] view whose last dim is contiguous."""
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a [tokens, heads, rope_dim] view, got {t.dim()} dims")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the rotary dims of a head must be contiguous")
    return t.stride(0), t.stride(1)


def rope_desc(x: torch.Tensor, out: torch.Tensor, flags: int = 0) -> RopeDesc:
    """Descriptor for turning x into out, [tokens, heads, rope_dim] views (slices of wider heads are
    fine; `out` may be `x`).  It holds for every pair of views of these shapes, strides and type."""
    if x.shape != out.shape or x.dtype != out.dtype:
        raise ValueError("x and out must have the same shape and dtype")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x: expected torch.bfloat16 or torch.float32, got {x.dtype}")
    xs, os_ = _heads_view(x, "x"), _heads_view(out, "out")
    return RopeDesc(x.shape[0], x.shape[1], x.shape[2], DSA_F32 if x.dtype == torch.float32 else DSA_BF16, xs[0], xs[1],
                    os_[0], os_[1], flags)


def _rope_view(t: torch.Tensor, dt, shape: tuple, token: int, head: int, name: str, dev: int) -> int:
    if t.dtype is not dt or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: expected a {dt} tensor of shape {shape} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    if t.stride() != (token, head, 1):
        s = _heads_view(t, name)        # (of one token or one head, the stride is never used)
        if (shape[0] > 1 and s[0] != token) or (shape[1] > 1 and s[1] != head):
            raise ValueError(f"{name}: strides {t.stride()} are not the descriptor's {(token, head)}")
    return t.data_ptr()


def dsa_rope_apply(desc: RopeDesc, x, pos, rope_cs, out, ws=None, stream=None) -> torch.Tensor:
    """out = x turned at pos (DSA_ROPE_INVERSE: by the negated angle, the gradient), [tokens, heads,
    rope_dim] views as the descriptor was made for."""
    n, r = desc.n_tokens, desc.rope_dim
    dt, shape = torch.float32 if desc.dtype == DSA_F32 else torch.bfloat16, (n, desc.n_heads, r)
    dev = _current_device(out, "out")
    px = _rope_view(x, dt, shape, desc.x_token_stride, desc.x_head_stride, "x", dev)
    po = _rope_view(out, dt, shape, desc.out_token_stride, desc.out_head_stride, "out", dev)
    n_pos = _rope_rows(rope_cs, r)
    if ws is None:
        ws = _workspace(256, out.device, stream)
    st = (_lib or lib()).dsa_rope_apply(desc, px, _arg(pos, torch.int32, n, "pos", dev),
                                        _arg(rope_cs, torch.float32, 0, "rope_cs", dev), n_pos, po,
                                        _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def _rope_rows(rope_cs: torch.Tensor, rope_dim: int) -> int:
    """Positions of a (cos, sin) table for rope_dim rotary dims."""
    s = rope_cs.shape
    if rope_cs.dtype is not torch.float32 or len(s) != 3 or s[1] != rope_dim // 2 or s[2] != 2:
        raise ValueError(f"rope_cs: expected a float32 [positions, {rope_dim // 2}, 2] tensor, got {rope_cs.dtype} "
                         f"{tuple(s)}")
    return s[0]


# ------------------------------------------------------------------------------ latent cache

def latent_cache(latent: torch.Tensor, scale: Optional[torch.Tensor] = None,
                 rope: Optional[torch.Tensor] = None) -> LatentCache:
    """A latent cache over the caller's tensors (kept alive by the caller): bf16 [n_rows, 576] alone,
    or fp8: codes [n_rows, 512] (uint8 or float8_e4m3fn), scale uint8 [n_rows, 4], rope bf16 [n_rows, 64]."""
    n = latent.shape[0]
    if scale is None and rope is None:
        if latent.dtype != torch.bfloat16 or latent.shape != (n, 576):
            raise ValueError(f"latent: expected bf16 [n_rows, 576], got {latent.dtype} {tuple(latent.shape)}")
        cache = LatentCache(_ptr(latent), None, None, n, DSA_CACHE_BF16)
        cache.device = latent.get_device()
        return cache
    if latent.dtype not in (torch.uint8, torch.float8_e4m3fn) or latent.shape != (n, 512):
        raise ValueError(f"latent: expected e4m3 codes [n_rows, 512], got {latent.dtype} {tuple(latent.shape)}")
    if scale is None or scale.dtype != torch.uint8 or scale.shape != (n, 4):
        raise ValueError("scale: expected uint8 [n_rows, 4]")
    if rope is None or rope.dtype != torch.bfloat16 or rope.shape != (n, 64):
        raise ValueError("rope: expected bf16 [n_rows, 64]")
    cache = LatentCache(_ptr(latent), _ptr(scale), _ptr(rope), n, DSA_CACHE_FP8)
    cache.device = _one_device(latent, scale, rope)
    return cache


def cache_write_desc(kv: torch.Tensor, flags: int = 0) -> CacheWriteDesc:
    """Descriptor for storing kv, a [tokens, 576] bf16 view with contiguous rows."""
    if kv.dtype != torch.bfloat16 or kv.dim() != 2 or kv.shape[1] != 576 or kv.stride(1) != 1:
        raise ValueError("kv: expected a bf16 [tokens, 576] view with contiguous rows")
    return CacheWriteDesc(kv.shape[0], flags, kv.stride(0) if kv.shape[0] > 1 else 576)


def dsa_latent_cache_write(desc: CacheWriteDesc, kv, slot, pos, rope_cs, cache: LatentCache, ws=None,
                           stream=None) -> torch.Tensor:
    """Store kv's rows in cache rows slot (negative: none), turned at pos with DSA_CACHE_ROPE."""
    n = desc.n_tokens
    if kv.dtype is not torch.bfloat16 or kv.shape != (n, 576) or kv.stride(1) != 1:
        raise ValueError(f"kv: expected a bf16 [{n}, 576] view with contiguous rows")
    if n > 1 and kv.stride(0) != desc.kv_stride:
        raise ValueError(f"kv: token stride {kv.stride(0)} is not the descriptor's {desc.kv_stride}")
    dev = _current_device(kv, "kv", cache)
    n_pos, p_pos, p_cs = 0, None, None
    if desc.flags & DSA_CACHE_ROPE:
        p_pos = _arg(pos, torch.int32, n, "pos", dev)
        n_pos, p_cs = _rope_rows(rope_cs, 64), _arg(rope_cs, torch.float32, 0, "rope_cs", dev)
    if ws is None:
        ws = _workspace(256, kv.device, stream)
    st = (_lib or lib()).dsa_latent_cache_write(desc, kv.data_ptr(), _arg(slot, torch.int32, n, "slot", dev), p_pos,
                                                p_cs, n_pos, cache, _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(),
                                                _stream(stream))
    if st:
        _check(st)
    return ws


def dsa_latent_cache_read(cache: LatentCache, pages: PagedCache, n_seq: int, row_start, kv_out, ws=None,
                          stream=None) -> torch.Tensor:
    """kv_out[row_start[t] + j] = row j of sequence t for every cached row of n_seq sequences, bf16."""
    _paged_args(pages, n_seq)
    s = kv_out.shape
    if len(s) != 2 or s[1] != 576:
        raise ValueError(f"kv_out: expected bf16 [rows, 576], got {kv_out.dtype} {tuple(s)}")
    dev = _current_device(kv_out, "kv_out", cache, pages)
    p_out = _arg(kv_out, torch.bfloat16, 0, "kv_out", dev)
    if ws is None:
        ws = _workspace(256, kv_out.device, stream)
    st = (_lib or lib()).dsa_latent_cache_read(cache, pages, n_seq,
                                               _arg(row_start, torch.int32, n_seq, "row_start", dev), p_out, s[0],
                                               _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def dsa_latent_attn_workspace_size(desc: AttnDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_latent_attn_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def dsa_latent_attn_paged(desc: AttnDesc, q, cache: LatentCache, idx, pages: PagedCache, out, lse=None, ws=None,
                          stream=None) -> torch.Tensor:
    """Latent attention of row t over its sequence's cached keys: all of them (idx None) or the
    selected ones."""
    n = desc.n_q * desc.n_heads
    dev = _current_device(q, "q", cache, pages)
    p_q, p_out = _arg(q, torch.bfloat16, n * desc.d_qk, "q", dev), _arg(out, torch.bfloat16, n * desc.d_v, "out", dev)
    p_idx = None if idx is None else _arg(idx, torch.int32, desc.n_q * desc.topk, "idx", dev)
    p_lse = None if lse is None else _arg(lse, torch.float32, n, "lse", dev)
    _paged_args(pages, desc.n_q)
    if ws is None:
        ws = _workspace(dsa_latent_attn_workspace_size(desc), q.device, stream)
    st = (_lib or lib()).dsa_latent_attn_paged(desc, p_q, cache, p_idx, pages, p_out, p_lse,
                                               _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def shared_rows(group_start: torch.Tensor, prefix_len: torch.Tensor, max_rows: int) -> SharedRows:
    """Groups of rows that share a prefix: rows [group_start[g], group_start[g + 1]) their first prefix_len[g]
    keys.  int32 device tensors of groups + 1 and of groups entries (kept alive by the caller); max_rows: rows of
    the largest group, or about."""
    n = prefix_len.numel()
    _want(group_start, torch.int32, n + 1, "group_start")
    _want(prefix_len, torch.int32, 0, "prefix_len")
    rows = SharedRows(_ptr(group_start), _ptr(prefix_len), n, max_rows)
    rows.device = _one_device(group_start, prefix_len)
    return rows


def dsa_latent_attn_shared_workspace_size(desc: AttnDesc, groups: SharedRows) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_latent_attn_shared_workspace_size(C.byref(desc), C.byref(groups), C.byref(n)))
    return n.value


def dsa_latent_attn_shared(desc: AttnDesc, q, cache: LatentCache, groups: SharedRows, pages: PagedCache, out, lse=None,
                           ws=None, stream=None) -> torch.Tensor:
    """Latent attention of row t over its sequence's cached keys, the keys that a group's rows share walked once
    for all of them."""
    n = desc.n_q * desc.n_heads
    dev = _current_device(q, "q", cache, groups, pages)
    p_q, p_out = _arg(q, torch.bfloat16, n * desc.d_qk, "q", dev), _arg(out, torch.bfloat16, n * desc.d_v, "out", dev)
    p_lse = None if lse is None else _arg(lse, torch.float32, n, "lse", dev)
    _paged_args(pages, desc.n_q)
    if ws is None:
        ws = _workspace(dsa_latent_attn_shared_workspace_size(desc, groups), q.device, stream)
    st = (_lib or lib()).dsa_latent_attn_shared(desc, p_q, cache, groups, pages, p_out, p_lse,
                                                _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def dsa_latent_key_weights_workspace_size(desc: AttnDesc, pages: PagedCache) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_latent_key_weights_workspace_size(C.byref(desc), C.byref(pages), C.byref(n)))
    return n.value


def _weight_rows(t: torch.Tensor, rows: int, width: int, name: str, dev: int) -> int:
    """Elements between the rows of a float32 [rows or more, width or more] view with contiguous rows."""
    if t.dtype is not torch.float32 or t.dim() != 2 or t.shape[0] < rows or t.shape[1] < width or t.get_device() != dev:
        raise ValueError(f"{name}: expected a float32 view of at least {(rows, width)} on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.stride(0) if rows > 1 else max(width, t.shape[1])


def dsa_latent_key_weights(desc: AttnDesc, q, cache: LatentCache, pages: PagedCache, lse, weight_in, weight_out,
                           ws=None, stream=None) -> torch.Tensor:
    """weight_out[t, j] = weight_in[t, j] (None: zeros) + the attention weights of key j over row t's heads.
    weight_in and weight_out: float32 [rows, max_pages * 128 or more] of the same row stride, or the same tensor."""
    n, width = desc.n_q, pages.max_pages * DSA_PAGE_ROWS
    dev = _current_device(q, "q", cache, pages)
    p_q, p_lse = (_arg(q, torch.bfloat16, n * desc.n_heads * desc.d_qk, "q", dev),
                  _arg(lse, torch.float32, n * desc.n_heads, "lse", dev))
    stride = _weight_rows(weight_out, n, width, "weight_out", dev)
    if weight_in is not None and _weight_rows(weight_in, n, width, "weight_in", dev) != stride and n > 1:
        raise ValueError("weight_in and weight_out must have the same row stride")
    _paged_args(pages, n)
    if ws is None:
        ws = _workspace(dsa_latent_key_weights_workspace_size(desc, pages), q.device, stream)
    st = (_lib or lib()).dsa_latent_key_weights(desc, p_q, cache, pages, p_lse,
                                                None if weight_in is None else weight_in.data_ptr(), weight_out.data_ptr(),
                                                stride, _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def evict_desc(n_seq: int, n_keep: int, n_first: int = 0, n_last: int = 0) -> EvictDesc:
    """n_keep keys of each longer sequence stay: the first n_first, the last n_last, the heaviest between."""
    return EvictDesc(n_seq, n_keep, n_first, n_last)


def dsa_latent_cache_evict_workspace_size(desc: EvictDesc) -> int:
    n = C.c_size_t(0)
    _check(lib().dsa_latent_cache_evict_workspace_size(C.byref(desc), C.byref(n)))
    return n.value


def dsa_latent_cache_evict(desc: EvictDesc, cache: LatentCache, pages: PagedCache, weight, to: LatentCache,
                           to_pages: PagedCache, kept, weight_out, new_len, ws=None, stream=None) -> torch.Tensor:
    """The heaviest keys of each sequence of `pages`, in order, copied to the rows of `to_pages`; kept[t]: their old
    positions, weight_out[t] (or None): their weights, new_len[t]: their number (to_pages' seq_len may be passed)."""
    n = desc.n_seq
    dev = _current_device(kept, "kept", cache, pages, to, to_pages)
    _paged_args(pages, n)
    _paged_args(to_pages, n)
    width = pages.max_pages * DSA_PAGE_ROWS
    stride = _weight_rows(weight, n, width, "weight", dev)
    out_stride = _weight_rows(weight_out, n, min(desc.n_keep, width), "weight_out", dev) if weight_out is not None else 0
    if ws is None:
        ws = _workspace(dsa_latent_cache_evict_workspace_size(desc), kept.device, stream)
    st = (_lib or lib()).dsa_latent_cache_evict(desc, cache, pages, weight.data_ptr(), stride, to, to_pages,
                                                _arg(kept, torch.int32, n * desc.n_keep, "kept", dev),
                                                None if weight_out is None else weight_out.data_ptr(), out_stride,
                                                _arg(new_len, torch.int32, n, "new_len", dev),
                                                _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def dsa_mtp_indexshare_step(idesc: IndexerDesc, adesc: AttnDesc, step: int, layer: dict, ks, ke, q_pos, k_pos,
                            rope_cs, mtp_idx, ws=None, stream=None):
    """One MTP draft step: step 0 runs the indexer into mtp_idx and attends with it; later
    steps attend with mtp_idx unchanged.  layer: 'q', 'kv', 'out' (+ 'lse') and, at step 0,
    'q_idx', 'k_idx', 'w'."""
    L = layer
    n_q, H, k = adesc.n_q, adesc.n_heads, adesc.topk
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for key, dt, n in (("q", bf, n_q * H * adesc.d_qk), ("kv", bf, adesc.n_kv * adesc.d_qk),
                       ("out", bf, n_q * H * adesc.d_v), ("lse", f32, n_q * H)):
        if L.get(key) is not None:
            _want(L[key], dt, n, key)
    _want(mtp_idx, i32, n_q * k, "mtp_idx")
    for t, dt, n, name in ((ks, i32, n_q, "ks"), (ke, i32, n_q, "ke"), (q_pos, i32, n_q, "q_pos")):
        _want(t, dt, n, name)
    if step == 0:
        _indexer_args(idesc, L.get("q_idx"), L.get("k_idx"), L.get("w"), None, k_pos, None, None, rope_cs, None, None)
    io = LayerIO(_ptr(L.get("q_idx")), _ptr(L.get("k_idx")), _ptr(L.get("w")), _ptr(L["q"]), _ptr(L["kv"]),
                 _ptr(L["out"]), _ptr(L.get("lse")))
    if ws is None:
        ws = _workspace(dsa_layers_workspace_size(idesc, adesc), L["q"].device, stream)
    n_pos = rope_cs.shape[0] if rope_cs is not None else 0
    _check(lib().dsa_mtp_indexshare_step(C.byref(idesc), C.byref(adesc), int(step), C.byref(io), _ptr(ks), _ptr(ke),
                                         _ptr(q_pos), _ptr(k_pos), _ptr(rope_cs), n_pos, _ptr(mtp_idx), _ptr(ws),
                                         ws.numel(), _stream(stream)))
    return ws


# ------------------------------------------------------------------------------ draft verification

def _vocab_rows(t: torch.Tensor, n: int, m: int, vocab: int, dt, name: str) -> int:
    """Elements between the vocabulary rows of a [n, m, vocab] view whose rows are equally far apart."""
    if t.dtype is not dt or t.shape != (n, m, vocab):
        raise ValueError(f"{name}: expected a {dt} view of shape {(n, m, vocab)}, got {t.dtype} {tuple(t.shape)}")
    s = t.stride()
    if vocab > 1 and s[2] != 1:
        raise ValueError(f"{name}: a row's probabilities must be contiguous")
    row = s[1] if m > 1 else s[0] if n > 1 else vocab
    if n > 1 and m > 1 and s[0] != m * row:
        raise ValueError(f"{name}: rows must be equally far apart, strides are {s}")
    return row


def verify_desc(target: torch.Tensor, draft: Optional[torch.Tensor] = None) -> VerifyDesc:
    """Descriptor for verifying drafts against target [sequences, drafts + 1, vocab], with the draft's
    probabilities [sequences, drafts, vocab] or without; fp32 or bf16 views whose rows are equally far apart.
    It holds for every pair of views of these shapes, strides and type."""
    if target.dim() != 3 or target.shape[1] < 1:
        raise ValueError(f"target: expected [sequences, drafts + 1, vocab], got {tuple(target.shape)}")
    if target.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"target: expected torch.bfloat16 or torch.float32, got {target.dtype}")
    n, m, v = target.shape
    row = _vocab_rows(target, n, m, v, target.dtype, "target")
    drow = _vocab_rows(draft, n, m - 1, v, target.dtype, "draft") if draft is not None else 0
    return VerifyDesc(n, m - 1, v, DSA_F32 if target.dtype == torch.float32 else DSA_BF16, row, drow)


def dsa_mtp_verify(desc: VerifyDesc, target, draft, tokens, draft_len, u_accept, u_sample, tokens_out, n_accepted,
                   ws=None, stream=None) -> torch.Tensor:
    """tokens_out[t] = the drafts of sequence t that are taken, the token drawn behind them, then -1;
    n_accepted[t] = how many were taken.  draft None: drafts without probabilities; draft_len None: all of them."""
    n, d, v = desc.n_seq, desc.n_draft, desc.vocab
    dt = torch.float32 if desc.dtype == DSA_F32 else torch.bfloat16
    dev = _current_device(target, "target")
    views = [(target, d + 1, desc.target_stride, "target")]
    if draft is not None and d > 0:
        views.append((draft, d, desc.draft_stride, "draft"))
    for t, m, row, name in views:
        if _vocab_rows(t, n, m, v, dt, name) != row:
            if n * m > 1:
                raise ValueError(f"{name}: strides {t.stride()} are not the descriptor's ({row} between rows)")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, but the call's other tensors are on cuda:{dev}")
    i32, f32 = torch.int32, torch.float32
    p_tok = p_u = None
    if d > 0:
        p_tok, p_u = _arg(tokens, i32, n * d, "tokens", dev), _arg(u_accept, f32, n * d, "u_accept", dev)
    p_len = None if draft_len is None else _arg(draft_len, i32, n, "draft_len", dev)
    if ws is None:
        ws = _workspace(256, target.device, stream)
    st = (_lib or lib()).dsa_mtp_verify(desc, target.data_ptr(), draft.data_ptr() if draft is not None else None, p_tok,
                                        p_len, p_u, _arg(u_sample, f32, n, "u_sample", dev),
                                        _arg(tokens_out, i32, n * (d + 1), "tokens_out", dev),
                                        _arg(n_accepted, i32, n, "n_accepted", dev),
                                        _arg(ws, torch.uint8, 0, "ws", dev), ws.numel(), _stream(stream))
    if st:
        _check(st)
    return ws


def dsa_workspace_status(ws: torch.Tensor, stream=None, raise_on_fault: bool = True) -> int:
    """Synchronise and read the device status bits of a workspace.

    Raises DsaError on a device fault unless raise_on_fault is False, in which case the raw
    bits are returned (0 = clean).  A CUDA error always raises.
    """
    bits = C.c_uint32(0)
    st = lib().dsa_workspace_status(_ptr(ws), _stream(stream), C.byref(bits))
    if st not in (0, 7, 8) or (st != 0 and raise_on_fault):
        _check(st)
    return bits.value


def dsa_profile_enable(on: bool) -> None:
    """Turn per-phase event recording of indexer calls on or off (process-wide)."""
    _check(lib().dsa_profile_enable(1 if on else 0))


def dsa_profile_indexer_last() -> list:
    """Device milliseconds of the last profiled indexer call on the current device:
    [RoPE, key-range plan, scores + streaming top-k, final select]."""
    ms = (C.c_float * 4)()
    _check(lib().dsa_profile_indexer_last(ms, 4))
    return [float(x) for x in ms]


def dsa_indexer_static_status(stream=None, raise_on_fault: bool = True) -> int:
    """Status bits of the last dsa_indexer_topk_static call on the current device (synchronises
    the stream).  Raises DsaError on a device fault unless raise_on_fault is False."""
    bits = C.c_uint32(0)
    st = lib().dsa_indexer_static_status(_stream(stream), C.byref(bits))
    if st not in (0, 7, 8) or (st != 0 and raise_on_fault):
        _check(st)
    return bits.value


def dsa_profile_read(cap: int = 8192) -> list:
    """[(kind name, device ms)] of every launch logged on the current device since profiling was
    switched on, in launch order (waits for them to finish)."""
    buf = (ProfileRecord * cap)()
    n = C.c_int32(0)
    _check(lib().dsa_profile_read(buf, cap, C.byref(n)))
    return [(PROFILE_KINDS.get(buf[i].kind, str(buf[i].kind)), float(buf[i].ms)) for i in range(min(n.value, cap))]


def dsa_debug_pipeline(stop_after_tiles: int = -1, wait_ns: int = 0) -> None:
    """Test hook: bound every pipeline wait at wait_ns (0: the default 2 s) and make the TMA
    producers stop after stop_after_tiles tiles (-1: never).  Process-wide."""
    _check(lib().dsa_debug_pipeline(int(stop_after_tiles), int(wait_ns)))
