"""GB300-native rotary position embedding: RoPE, M-RoPE, on-the-fly RoPE.

A thin binding over the C ABI of ``librope_gb300.so`` (``include/rope.h``).
This module only marshals arguments -- tensor pointers, shapes, attributes,
the current CUDA stream -- and allocates outputs the way the operators' own
JavaScript API does; every step of the computation runs in the library's
CUDA kernels. PyTorch supplies device memory and streams.

There is no CPU fallback: if the library cannot be loaded, every call raises.
"""

import ctypes
import os
import threading

from .build import BINDING_PATH, LIB_PATH, build_library  # noqa: F401

__all__ = [
    "RopeError", "load_library", "build_library", "rope_apply", "mrope_apply",
    "mrope_apply_stream_map", "mrope_stream_map", "rope_apply_fused", "rope_cache_build",
    "rope_apply_qkv", "mrope_apply_qkv", "rope_apply_qkv_fp8", "kv_attention", "kv_attention_fp8",
    "kv_attention_workspace", "kv_cache_fp8",
    "rope_apply_qkv_paged", "kv_attention_paged", "kv_attention_paged_workspace", "kv_keep_paged", "kv_cache_paged",
    "set_variant", "get_variant", "variant",
    "ROPE_OK", "ROPE_ERR_INVALID_ARG", "ROPE_ERR_UNSUPPORTED", "ROPE_ERR_CUDA",
]

ROPE_OK, ROPE_ERR_INVALID_ARG, ROPE_ERR_UNSUPPORTED, ROPE_ERR_CUDA = 0, 1, 2, 3
ROPE_F32, ROPE_F16, ROPE_BF16 = 0, 1, 2
ROPE_SCRATCH_BYTES = 64
ROPE_KV_SCALE_BLOCK = 16
VARIANTS = {"auto": 0, "simt": 1, "tma": 2}
_UNSUPPORTED_DTYPE = 99  # passed through so the library reports ROPE_ERR_UNSUPPORTED

_lock = threading.Lock()
_lib = None
_short = None  # csrc/binding.cpp once it was asked for, or False

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_i64p = ctypes.POINTER(ctypes.c_int64)
_i32p = ctypes.POINTER(ctypes.c_int32)
_u8p = ctypes.POINTER(ctypes.c_uint8)

# name -> argtypes (restype is the int status unless listed in _RESTYPES)
SIGNATURES = {
    "rope_apply": [_i32, _i32, _i64p, _vp, _vp, _i32, _i64p, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                   _vp],
    "mrope_apply": [_i32, _i32, _i64p, _vp, _vp, _i64, _vp, _vp, _vp, _i32p, _i32, _f32, _i32, _i32,
                    _i32, _i32, _vp, _vp, _vp],
    "mrope_apply_stream_map": [_i32, _i32, _i64p, _vp, _vp, _i64, _vp, _vp, _vp, _u8p, _f32, _i32,
                               _i32, _i32, _vp, _vp, _vp],
    "mrope_stream_map": [_i32p, _i32, _i32, _u8p],
    "rope_apply_fused": [_i32, _i32, _i64p, _vp, _vp, _vp, _f32, _vp, _i32, _i32, _i32, _vp],
    "mrope_apply_fused": [_i32, _i32, _i64p, _vp, _vp, _vp, _f32, _vp, _i32p, _i32, _f32, _i32, _i32, _i32, _vp],
    "rope_cache_build": [_i32, _vp, _i32, _i64, _f32, _vp, _vp, _vp],
    "rope_apply_qkv": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _i32,
                       _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp],
    "rope_apply_qkv_rmsnorm": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp,
                               _i64, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp],
    "mrope_apply_qkv": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _i64, _vp,
                        _i32p, _i32, _f32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp],
    "rope_apply_no_alloc": [_i32, _i32, _i64p, _vp, _vp, _i32, _i64p, _vp, _vp, _vp, _i32, _i32, _i32, _vp,
                            _vp],
    "rope_apply_qkv_fp8": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _i64,
                           _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp],
    "kv_attention": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _i64, _vp, _f32, _f32, _vp, _vp, _vp,
                     _vp, _vp, _vp, _i64, _vp],
    "kv_attention_fp8": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _f32, _f32, _vp,
                         _vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "kv_attention_workspace": [_i64, _i64, _i32, _i32, _i64, _i64],
    "rope_apply_qkv_paged": [_i32, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _i64, _vp,
                             _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp],
    "kv_attention_paged": [_i32, _i64, _i64, _i64, _i32, _i32, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp,
                           _vp, _f32, _f32, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "kv_attention_paged_workspace": [_i32, _i64, _i64, _i64, _i32, _i32, _i64, _i64, _i64],
    "kv_keep_paged": [_i32, _i64, _i32, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp],
    "rope_set_variant": [_i32],
    "rope_get_variant": [],
    "rope_status_string": [_i32],
    "rope_last_error": [],
    "rope_last_kernel": [],
}
_RESTYPES = {"rope_status_string": ctypes.c_char_p, "rope_last_error": ctypes.c_char_p,
             "rope_last_kernel": ctypes.c_char_p, "kv_attention_workspace": _i64,
             "kv_attention_paged_workspace": _i64}


class RopeError(RuntimeError):
    def __init__(self, fn, status, message):
        self.status = status
        self.message = message
        names = {1: "ROPE_ERR_INVALID_ARG", 2: "ROPE_ERR_UNSUPPORTED", 3: "ROPE_ERR_CUDA"}
        super().__init__(f"{fn}: {names.get(status, status)}: {message}")


def load_library(path=None):
    """Load librope_gb300.so (built in-tree by ``build_library()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"librope_gb300.so not found at {p}: run "
                "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc); "
                "there is no CPU fallback")
        lib = ctypes.CDLL(p)
        for name, args in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = _RESTYPES.get(name, ctypes.c_int)
        if path is None:
            _lib = lib
        return lib


def _short_way():
    """csrc/binding.cpp's module, bound to the library, or False where it was not compiled."""
    global _short
    if _short is None:
        lib = load_library()
        with _lock:
            if _short is None:
                module = False
                if os.path.exists(BINDING_PATH):
                    import importlib.machinery
                    import importlib.util

                    import torch  # noqa: F401  (its libraries are what the module links to)

                    name = __name__ + "._binding"
                    loader = importlib.machinery.ExtensionFileLoader(name, BINDING_PATH)
                    spec = importlib.util.spec_from_file_location(name, BINDING_PATH, loader=loader)
                    try:
                        module = importlib.util.module_from_spec(spec)
                        loader.exec_module(module)
                        module.bind(*[ctypes.cast(getattr(lib, fn), _vp).value for fn in (
                            "rope_apply_qkv_paged", "kv_attention_paged", "kv_attention_paged_workspace",
                            "kv_keep_paged")])
                    except ImportError:  # compiled for another PyTorch or machine
                        module = False
                _short = module
    return _short


def _check(fn, status):
    if status != ROPE_OK:
        msg = load_library().rope_last_error().decode()
        raise RopeError(fn, status, msg)


# --------------------------------------------------------------------------
# marshalling helpers (torch is imported lazily: the host-only helpers work
# without it)
# --------------------------------------------------------------------------

def _dtype_code(t):
    import torch

    return {torch.float32: ROPE_F32, torch.float16: ROPE_F16, torch.bfloat16: ROPE_BF16}.get(
        t.dtype, _UNSUPPORTED_DTYPE)


def _shape(t):
    return (ctypes.c_int64 * max(1, t.dim()))(*[int(d) for d in t.shape])


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(name, t, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    return t


def _stream(x, stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    return ctypes.c_void_p(s.cuda_stream)


_scratch = {}


def _scratch_ptr(x, stream, scratch):
    """The scratch argument: None (default) -> the static schedule; a tensor ->
    that buffer (ROPE_SCRATCH_BYTES, zeroed before its first use); "auto" -> one
    zeroed buffer per (device, stream), owned by this module, so launches on one
    stream share it and streams never do."""
    import torch

    if scratch is None or scratch is False:
        return None
    if isinstance(scratch, torch.Tensor):
        _cuda("scratch", scratch)
        if scratch.numel() * scratch.element_size() < ROPE_SCRATCH_BYTES:
            raise ValueError(f"scratch needs {ROPE_SCRATCH_BYTES} bytes")
        return ctypes.c_void_p(scratch.data_ptr())
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    key = (x.device.index, s.cuda_stream)
    buf = _scratch.get(key)
    if buf is None:
        buf = torch.zeros(ROPE_SCRATCH_BYTES // 8, dtype=torch.int64, device=x.device)
        _scratch[key] = buf
    return ctypes.c_void_p(buf.data_ptr())


def _out(x, out):
    import torch

    if out is None:
        return torch.empty_like(x)
    _cuda("out", out, x.dtype)
    if out.shape != x.shape:
        raise ValueError(f"out shape {tuple(out.shape)} != x shape {tuple(x.shape)}")
    return out


# --------------------------------------------------------------------------
# public API (same names as the C ABI)
# --------------------------------------------------------------------------

def rope_apply(x, cos_cache, sin_cache, position_ids=None, *, interleaved=0, rotary_embedding_dim=0,
               num_heads=0, out=None, oor_flag=None, stream=None, scratch=None):
    """RotaryEmbedding (see ``rope_apply`` in include/rope.h). Returns Y."""
    import torch

    lib = load_library()
    _cuda("x", x)
    _cuda("cos_cache", cos_cache)
    _cuda("sin_cache", sin_cache)
    _cuda("position_ids", position_ids, torch.int64)
    _cuda("oor_flag", oor_flag, torch.int32)
    y = _out(x, out)
    with torch.cuda.device(x.device):
        st = lib.rope_apply(_dtype_code(x), x.dim(), _shape(x), _ptr(x), _ptr(y), cos_cache.dim(),
                            _shape(cos_cache), _ptr(cos_cache), _ptr(sin_cache), _ptr(position_ids),
                            int(interleaved), int(rotary_embedding_dim), int(num_heads), _ptr(oor_flag),
                            _scratch_ptr(x, stream, scratch), _stream(x, stream))
    _check("rope_apply", st)
    return y


def mrope_apply(x, cos_cache, sin_cache, position_ids, mrope_section, *, mrope_layout=0, scale=1.0,
                interleaved=0, rotary_embedding_dim=0, num_heads=0, is_packed_batching=0, out=None,
                oor_flag=None, stream=None, scratch=None):
    """MRotaryEmbedding (see ``mrope_apply`` in include/rope.h). Returns Y."""
    import torch

    lib = load_library()
    _cuda("x", x)
    _cuda("cos_cache", cos_cache)
    _cuda("sin_cache", sin_cache)
    _cuda("position_ids", position_ids, torch.int64)
    _cuda("oor_flag", oor_flag, torch.int32)
    y = _out(x, out)
    sec = (ctypes.c_int32 * 3)(*[int(v) for v in mrope_section])
    with torch.cuda.device(x.device):
        st = lib.mrope_apply(_dtype_code(x), x.dim(), _shape(x), _ptr(x), _ptr(y), int(cos_cache.shape[0]),
                             _ptr(cos_cache), _ptr(sin_cache), _ptr(position_ids), sec, int(mrope_layout),
                             float(scale), int(interleaved), int(rotary_embedding_dim), int(num_heads),
                             int(is_packed_batching), _ptr(oor_flag), _scratch_ptr(x, stream, scratch),
                             _stream(x, stream))
    _check("mrope_apply", st)
    return y


def mrope_apply_stream_map(x, cos_cache, sin_cache, position_ids, stream_map, *, scale=1.0, interleaved=0,
                           rotary_embedding_dim=0, num_heads=0, out=None, oor_flag=None, stream=None,
                           scratch=None):
    """MRotaryEmbedding with an explicit stream (0 t, 1 h, 2 w) per half-rotary index."""
    import torch

    lib = load_library()
    _cuda("x", x)
    _cuda("cos_cache", cos_cache)
    _cuda("sin_cache", sin_cache)
    _cuda("position_ids", position_ids, torch.int64)
    _cuda("oor_flag", oor_flag, torch.int32)
    y = _out(x, out)
    m = list(int(v) for v in stream_map)
    arr = (ctypes.c_uint8 * max(1, len(m)))(*m)
    with torch.cuda.device(x.device):
        st = lib.mrope_apply_stream_map(_dtype_code(x), x.dim(), _shape(x), _ptr(x), _ptr(y),
                                        int(cos_cache.shape[0]), _ptr(cos_cache), _ptr(sin_cache),
                                        _ptr(position_ids), arr, float(scale), int(interleaved),
                                        int(rotary_embedding_dim), int(num_heads), _ptr(oor_flag),
                                        _scratch_ptr(x, stream, scratch), _stream(x, stream))
    _check("mrope_apply_stream_map", st)
    return y


def mrope_stream_map(mrope_section, mrope_layout, half):
    """Host helper: the stream of each half-rotary index, as mrope_apply uses it."""
    lib = load_library()
    sec = (ctypes.c_int32 * 3)(*[int(v) for v in mrope_section])
    out = (ctypes.c_uint8 * max(1, int(half)))()
    _check("mrope_stream_map", lib.mrope_stream_map(sec, int(mrope_layout), int(half), out))
    return list(out)[: int(half)]


def rope_apply_fused(x, inv_freq, position_ids, *, attention_scaling=1.0, interleaved=0,
                     rotary_embedding_dim=0, num_heads=0, out=None, stream=None):
    """RotaryEmbedding with cos/sin computed on the fly from inv_freq."""
    import torch

    lib = load_library()
    _cuda("x", x)
    _cuda("inv_freq", inv_freq, torch.float32)
    _cuda("position_ids", position_ids, torch.int64)
    y = _out(x, out)
    with torch.cuda.device(x.device):
        st = lib.rope_apply_fused(_dtype_code(x), x.dim(), _shape(x), _ptr(x), _ptr(y), _ptr(inv_freq),
                                  float(attention_scaling), _ptr(position_ids), int(interleaved),
                                  int(rotary_embedding_dim), int(num_heads), _stream(x, stream))
    _check("rope_apply_fused", st)
    return y


def rope_apply_qkv(query, cos_cache, sin_cache, position_ids=None, *, num_heads, kv_num_heads, key=None,
                   value=None, interleaved=0, rotary_embedding_dim=0, k_cache=None, v_cache=None,
                   past_seq_lens=None, q_out=None, k_out=None, status=None, q_norm_weight=None,
                   k_norm_weight=None, epsilon=1e-6, stream=None, scratch=None):
    """Q and K rotation for grouped-query attention in one launch, optionally
    appending rotated K and V to (B, kv_num_heads, max_len, H) caches in place.
    With q_norm_weight and k_norm_weight (head_size vectors) each Q and K head
    is RMS-normalised first (rope_apply_qkv_rmsnorm).

    query is (B, S, num_heads*H), or packed [Q|K|V] (B, S, (num_heads +
    2*kv_num_heads)*H) when key and value are None. Returns (q_out, k_out);
    k_out is None in cache mode (the caches hold the result). scratch: None,
    or ROPE_SCRATCH_BYTES of zeroed device memory for the dynamic tile schedule
    (one per concurrently running stream).
    """
    import torch

    lib = load_library()
    _cuda("query", query)
    for name, t in (("key", key), ("value", value), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("cos_cache", cos_cache), ("sin_cache", sin_cache)):
        _cuda(name, t, query.dtype)
    _cuda("position_ids", position_ids, torch.int64)
    _cuda("past_seq_lens", past_seq_lens, torch.int32)
    if query.dim() != 3:
        raise ValueError("query must be (B, S, hidden)")
    B, S, hidden = query.shape
    packed = key is None and value is None
    rows_per_tok = num_heads + (2 * kv_num_heads if packed else 0)
    if hidden % rows_per_tok:
        raise ValueError(f"query hidden size {hidden} is not a multiple of {rows_per_tok} heads")
    H = hidden // rows_per_tok
    if q_out is None:
        q_out = torch.empty((B, S, num_heads * H), dtype=query.dtype, device=query.device)
    cache = k_cache is not None
    if not cache and k_out is None:
        k_out = torch.empty((B, S, kv_num_heads * H), dtype=query.dtype, device=query.device)
    max_len = k_cache.shape[2] if cache else 0
    norm = q_norm_weight is not None or k_norm_weight is not None
    _cuda("q_norm_weight", q_norm_weight, query.dtype)
    _cuda("k_norm_weight", k_norm_weight, query.dtype)
    with torch.cuda.device(query.device):
        if norm:
            st = lib.rope_apply_qkv_rmsnorm(
                _dtype_code(query), B, S, int(num_heads), int(kv_num_heads), H, _ptr(query), _ptr(key),
                _ptr(value), _ptr(q_norm_weight), _ptr(k_norm_weight), float(epsilon), _ptr(cos_cache),
                _ptr(sin_cache), int(cos_cache.shape[0]), _ptr(position_ids), _ptr(past_seq_lens),
                int(interleaved), int(rotary_embedding_dim), _ptr(q_out), _ptr(k_out), _ptr(k_cache),
                _ptr(v_cache), int(max_len), _ptr(status), _ptr(scratch), _stream(query, stream))
        else:
            st = lib.rope_apply_qkv(_dtype_code(query), B, S, int(num_heads), int(kv_num_heads), H, _ptr(query),
                                    _ptr(key), _ptr(value), _ptr(cos_cache), _ptr(sin_cache),
                                    int(cos_cache.shape[0]), _ptr(position_ids), _ptr(past_seq_lens),
                                    int(interleaved), int(rotary_embedding_dim), _ptr(q_out), _ptr(k_out),
                                    _ptr(k_cache), _ptr(v_cache), int(max_len), _ptr(status), _ptr(scratch),
                                    _stream(query, stream))
    _check("rope_apply_qkv_rmsnorm" if norm else "rope_apply_qkv", st)
    return q_out, (None if cache else k_out)


def mrope_apply_qkv(query, cos_cache, sin_cache, position_ids, mrope_section, *, num_heads, kv_num_heads,
                    mrope_layout=0, scale=1.0, key=None, value=None, interleaved=0, rotary_embedding_dim=0,
                    k_cache=None, v_cache=None, past_seq_lens=None, q_out=None, k_out=None, status=None,
                    q_norm_weight=None, k_norm_weight=None, epsilon=1e-6, stream=None, scratch=None):
    """rope_apply_qkv with M-RoPE: position_ids is (3, B, S) (t, h, w) and every Q and K
    head is rotated as mrope_apply rotates a head; optional QK-RMSNorm first. Returns
    (q_out, k_out); k_out is None in cache mode."""
    import torch

    lib = load_library()
    _cuda("query", query)
    for name, t in (("key", key), ("value", value), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("cos_cache", cos_cache), ("sin_cache", sin_cache), ("q_norm_weight", q_norm_weight),
                    ("k_norm_weight", k_norm_weight)):
        _cuda(name, t, query.dtype)
    _cuda("position_ids", position_ids, torch.int64)
    _cuda("past_seq_lens", past_seq_lens, torch.int32)
    if query.dim() != 3:
        raise ValueError("query must be (B, S, hidden)")
    B, S, hidden = query.shape
    packed = key is None and value is None
    rows_per_tok = num_heads + (2 * kv_num_heads if packed else 0)
    if hidden % rows_per_tok:
        raise ValueError(f"query hidden size {hidden} is not a multiple of {rows_per_tok} heads")
    H = hidden // rows_per_tok
    if q_out is None:
        q_out = torch.empty((B, S, num_heads * H), dtype=query.dtype, device=query.device)
    cache = k_cache is not None
    if not cache and k_out is None:
        k_out = torch.empty((B, S, kv_num_heads * H), dtype=query.dtype, device=query.device)
    max_len = k_cache.shape[2] if cache else 0
    sec = (ctypes.c_int32 * 3)(*[int(v) for v in mrope_section])
    with torch.cuda.device(query.device):
        st = lib.mrope_apply_qkv(_dtype_code(query), B, S, int(num_heads), int(kv_num_heads), H, _ptr(query),
                                 _ptr(key), _ptr(value), _ptr(q_norm_weight), _ptr(k_norm_weight), float(epsilon),
                                 _ptr(cos_cache), _ptr(sin_cache), int(cos_cache.shape[0]), _ptr(position_ids),
                                 sec, int(mrope_layout), float(scale), _ptr(past_seq_lens), int(interleaved),
                                 int(rotary_embedding_dim), _ptr(q_out), _ptr(k_out), _ptr(k_cache), _ptr(v_cache),
                                 int(max_len), _ptr(status), _ptr(scratch), _stream(query, stream))
    _check("mrope_apply_qkv", st)
    return q_out, (None if cache else k_out)


def mrope_apply_fused(x, inv_freq, position_ids, mrope_section, *, mrope_layout=0, scale=1.0,
                      attention_scaling=1.0, interleaved=0, rotary_embedding_dim=0, num_heads=0, out=None,
                      stream=None):
    """MRotaryEmbedding with cos/sin computed on the fly from inv_freq (three position streams)."""
    import torch

    lib = load_library()
    _cuda("x", x)
    _cuda("inv_freq", inv_freq, torch.float32)
    _cuda("position_ids", position_ids, torch.int64)
    y = _out(x, out)
    sec = (ctypes.c_int32 * 3)(*[int(v) for v in mrope_section])
    with torch.cuda.device(x.device):
        st = lib.mrope_apply_fused(_dtype_code(x), x.dim(), _shape(x), _ptr(x), _ptr(y), _ptr(inv_freq),
                                   float(attention_scaling), _ptr(position_ids), sec, int(mrope_layout),
                                   float(scale), int(interleaved), int(rotary_embedding_dim), int(num_heads),
                                   _stream(x, stream))
    _check("mrope_apply_fused", st)
    return y


def rope_cache_build(inv_freq, rows, dtype=None, *, attention_scaling=1.0, cos_out=None, sin_out=None,
                     stream=None):
    """(rows, len(inv_freq)) cos and sin tables. Returns (cos, sin)."""
    import torch

    lib = load_library()
    _cuda("inv_freq", inv_freq, torch.float32)
    dtype = dtype or torch.float16
    half = int(inv_freq.shape[0])
    if cos_out is None:
        cos_out = torch.empty((int(rows), half), dtype=dtype, device=inv_freq.device)
    if sin_out is None:
        sin_out = torch.empty((int(rows), half), dtype=dtype, device=inv_freq.device)
    _cuda("cos_out", cos_out, dtype)
    _cuda("sin_out", sin_out, dtype)
    code = _dtype_code(cos_out)
    with torch.cuda.device(inv_freq.device):
        st = lib.rope_cache_build(code, _ptr(inv_freq), half, int(rows), float(attention_scaling),
                                  _ptr(cos_out), _ptr(sin_out), _stream(inv_freq, stream))
    _check("rope_cache_build", st)
    return cos_out, sin_out


# --------------------------------------------------------------------------
# 8-bit caches and attention over the caches
# --------------------------------------------------------------------------

def _shaped(name, t, like, shape, *dtypes):
    """``t`` checked: contiguous, on the device of ``like``, of one of the dtypes and of the shape."""
    if t is None:
        return None
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name} must be a CUDA tensor on {like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _address(t):
    return None if t is None else t.data_ptr()


def _fits(t, index, shape, dtype):
    """Whether ``t`` is what ``_shaped`` asks for, on CUDA device ``index`` (that one says what is wrong)."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


class _on:
    """The device current and, where the caller names one, ``stream`` too, so that what is allocated
    belongs to the stream that the launch runs on."""

    def __init__(self, dev, stream):
        import torch

        self.was = [torch.cuda.device(dev)]
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream must be one of {dev}, got {stream}")
            self.was.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.was:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.was):
            c.__exit__(*exc)


def _elsewhere(torch, dev, stream):
    """Whether a call has to change the current device or stream (see ``_on``)."""
    return stream is not None or dev.index != torch._C._cuda_getDevice()


_codes_of = {}


def _torch_code(T):
    """(torch, the C ABI's code of dtype T); torch is imported at the first call."""
    code = _codes_of.get(T)
    if code is None:
        import torch

        _codes_of.update({torch.float32: (torch, ROPE_F32), torch.float16: (torch, ROPE_F16),
                          torch.bfloat16: (torch, ROPE_BF16)})
        code = _codes_of.get(T, (torch, _UNSUPPORTED_DTYPE))
    return code


def kv_cache_fp8(batch, kv_num_heads, max_cache_len, head_size, device=None):
    """Empty 8-bit caches for rope_apply_qkv_fp8: (k_cache, v_cache, k_scale, v_scale). Codes are
    float8_e4m3fn (batch, kv_num_heads, max_cache_len, head_size), scales float32 with one value for
    ROPE_KV_SCALE_BLOCK rows of a head."""
    import torch

    device = torch.device("cuda") if device is None else device
    blocks = -(-max_cache_len // ROPE_KV_SCALE_BLOCK)
    codes = [torch.zeros((batch, kv_num_heads, max_cache_len, head_size), dtype=torch.uint8,
                         device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((batch, kv_num_heads, blocks), dtype=torch.float32, device=device) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def rope_apply_qkv_fp8(query, cos_cache, sin_cache, position_ids=None, *, num_heads, kv_num_heads, k_cache, v_cache,
                       k_scale, v_scale, past_seq_lens, key=None, value=None, interleaved=0, rotary_embedding_dim=0,
                       q_out=None, status=None, q_norm_weight=None, k_norm_weight=None, epsilon=1e-6, stream=None):
    """rope_apply_qkv in cache mode with caches held in 8 bits (see ``rope_apply_qkv_fp8`` in include/rope.h).

    k_cache and v_cache are float8_e4m3fn (or uint8 codes) (B, kv_num_heads, max_len, H), k_scale and v_scale
    float32 (B, kv_num_heads, ceil(max_len / 16)), all updated in place (``kv_cache_fp8`` makes them). With
    q_norm_weight and k_norm_weight each Q and K head is RMS-normalised first. Returns q_out."""
    lib = load_library()
    T, dev = query.dtype, query.device
    torch, code = _torch_code(T)
    if query.dim() != 3:
        raise ValueError("query must be (B, S, hidden)")
    B, S, hidden = query.shape
    packed = key is None and value is None
    rows_per_tok = num_heads + (2 * kv_num_heads if packed else 0)
    if rows_per_tok < 1 or hidden % rows_per_tok:
        raise ValueError(f"query hidden size {hidden} is not a multiple of {rows_per_tok} heads")
    H = hidden // rows_per_tok
    if k_cache.dim() != 4 or cos_cache.dim() != 2:
        raise ValueError("k_cache must be (B, kv_num_heads, max_len, H) and cos_cache (rows, rd/2)")
    L = k_cache.shape[2]
    plane = (B, kv_num_heads, L, H)
    blocks = (B, kv_num_heads, -(-L // ROPE_KV_SCALE_BLOCK))
    table = (cos_cache.shape[0], (rotary_embedding_dim or H) // 2)
    f32, kind, at = torch.float32, k_cache.dtype, query.get_device()
    if past_seq_lens is None or at < 0 or not (
            _fits(past_seq_lens, at, (B,), torch.int32) and _fits(k_cache, at, plane, kind)
            and _fits(v_cache, at, plane, kind) and _fits(k_scale, at, blocks, f32)
            and _fits(v_scale, at, blocks, f32) and _fits(cos_cache, at, table, T) and _fits(sin_cache, at, table, T)
            and query.is_contiguous()):
        codes = (torch.float8_e4m3fn, torch.uint8)
        _shaped("query", query, query, query.shape, T)
        _shaped("past_seq_lens", past_seq_lens, query, (B,), torch.int32)
        _shaped("k_cache", k_cache, query, plane, *codes)
        _shaped("v_cache", v_cache, query, plane, kind)
        _shaped("k_scale", k_scale, query, blocks, f32)
        _shaped("v_scale", v_scale, query, blocks, f32)
        _shaped("cos_cache", cos_cache, query, table, T)
        _shaped("sin_cache", sin_cache, query, table, T)
    if kind is not torch.float8_e4m3fn and kind is not torch.uint8:
        raise ValueError(f"k_cache must have dtype float8_e4m3fn or uint8, got {kind}")
    if not packed:
        _shaped("key", key, query, (B, S, kv_num_heads * H), T)
        _shaped("value", value, query, (B, S, kv_num_heads * H), T)
    if q_norm_weight is not None or k_norm_weight is not None:
        _shaped("q_norm_weight", q_norm_weight, query, (H,), T)
        _shaped("k_norm_weight", k_norm_weight, query, (H,), T)
    if position_ids is not None:
        _shaped("position_ids", position_ids, query, (B, S), torch.int64)
    if q_out is not None:
        _shaped("q_out", q_out, query, (B, S, num_heads * H), T)
    if status is not None:
        _shaped("status", status, query, status.shape, torch.int32)
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return rope_apply_qkv_fp8(
                query, cos_cache, sin_cache, position_ids, num_heads=num_heads, kv_num_heads=kv_num_heads,
                k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, past_seq_lens=past_seq_lens,
                key=key, value=value, interleaved=interleaved, rotary_embedding_dim=rotary_embedding_dim, q_out=q_out,
                status=status, q_norm_weight=q_norm_weight, k_norm_weight=k_norm_weight, epsilon=epsilon)
    if q_out is None:
        q_out = torch.empty((B, S, num_heads * H), dtype=T, device=dev)
    st = lib.rope_apply_qkv_fp8(
        code, B, S, num_heads, kv_num_heads, H, query.data_ptr(), _address(key), _address(value),
        _address(q_norm_weight), _address(k_norm_weight), epsilon, cos_cache.data_ptr(), sin_cache.data_ptr(),
        table[0], _address(position_ids), _address(past_seq_lens), int(interleaved), rotary_embedding_dim,
        q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), L,
        _address(status), torch._C._cuda_getCurrentRawStream(at))
    if st:
        _check("rope_apply_qkv_fp8", st)
    return q_out


def kv_attention_workspace(batch, seq, num_heads, kv_num_heads, head_size, max_cache_len):
    """Bytes of workspace that kv_attention and kv_attention_fp8 use for such a call."""
    n = load_library().kv_attention_workspace(batch, seq, num_heads, kv_num_heads, head_size, max_cache_len)
    if n < 0:
        _check("kv_attention_workspace", ROPE_ERR_INVALID_ARG)
    return n


_workspace_bytes = {}


def _workspace(fn, key):
    """A call's workspace by its sizes, asked for once (it follows from them and the variant); each function
    has keys of a length of its own."""
    n = _workspace_bytes.get(key)
    if n is None:
        if len(_workspace_bytes) > 4096:
            _workspace_bytes.clear()
        n = _workspace_bytes[key] = fn(*key)
    return n


def _attention(name, query, k_cache, v_cache, scales, past_seq_lens, num_heads, scale, softcap, alibi_slopes,
               document_ids, prefix_lens, out, status, workspace, stream):
    lib = load_library()
    T, dev, at, kind, plane = query.dtype, query.device, query.get_device(), k_cache.dtype, k_cache.shape
    torch, code = _torch_code(T)
    if query.dim() != 3 or len(plane) != 4:
        raise ValueError("query must be (B, S, num_heads*H) and k_cache (B, kv_num_heads, max_len, H)")
    B, S, hidden = query.shape
    _, N, L, H = plane
    f32, i32 = torch.float32, torch.int32
    ks = vs = None
    if scales is not None:
        ks, vs = scales
        blocks = (B, N, -(-L // ROPE_KV_SCALE_BLOCK))
        if ks is None or vs is None or not (_fits(ks, at, blocks, f32) and _fits(vs, at, blocks, f32)):
            _shaped("k_scale", ks, query, blocks, f32)
            _shaped("v_scale", vs, query, blocks, f32)
    if past_seq_lens is None or at < 0 or not (
            hidden == num_heads * H and plane[0] == B and query.is_contiguous() and _fits(past_seq_lens, at, (B,), i32)
            and _fits(k_cache, at, plane, kind) and _fits(v_cache, at, plane, kind)):
        _shaped("query", query, query, (B, S, num_heads * H), T)
        _shaped("k_cache", k_cache, query, (B, N, L, H), kind)
        _shaped("v_cache", v_cache, query, (B, N, L, H), kind)
        _shaped("past_seq_lens", past_seq_lens, query, (B,), i32)
    if kind is not T if scales is None else kind is not torch.float8_e4m3fn and kind is not torch.uint8:
        raise ValueError(f"k_cache must have dtype {T if scales is None else 'float8_e4m3fn or uint8'}, got {kind}")
    if alibi_slopes is not None:
        _shaped("alibi_slopes", alibi_slopes, query, (num_heads,), f32)
    if document_ids is not None:
        _shaped("document_ids", document_ids, query, (B, L), i32)
    if prefix_lens is not None:
        _shaped("prefix_lens", prefix_lens, query, (B,), i32)
    if out is not None:
        _shaped("out", out, query, (B, S, hidden), T)
    if status is not None:
        _shaped("status", status, query, status.shape, i32)
    if workspace is not None:
        _shaped("workspace", workspace, query, workspace.shape, torch.uint8)
    if scale is None:
        scale = max(H, 1) ** -0.5
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return _attention(name, query, k_cache, v_cache, scales, past_seq_lens, num_heads, scale, softcap,
                              alibi_slopes, document_ids, prefix_lens, out, status, workspace, None)
    if out is None:
        out = torch.empty_like(query)
    if workspace is None:
        need = _workspace(lib.kv_attention_workspace, (B, S, num_heads, N, H, L))
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    room = 0 if workspace is None else workspace.numel()
    handle = torch._C._cuda_getCurrentRawStream(at)
    if scales is None:
        st = lib.kv_attention(code, B, S, num_heads, N, H, query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), L,
                              _address(past_seq_lens), scale, softcap, _address(alibi_slopes), _address(document_ids),
                              _address(prefix_lens), out.data_ptr(), _address(status), _address(workspace), room,
                              handle)
    else:
        st = lib.kv_attention_fp8(code, B, S, num_heads, N, H, query.data_ptr(), k_cache.data_ptr(),
                                  v_cache.data_ptr(), _address(ks), _address(vs), L, _address(past_seq_lens), scale,
                                  softcap, _address(alibi_slopes), _address(document_ids), _address(prefix_lens),
                                  out.data_ptr(), _address(status), _address(workspace), room, handle)
    if st:
        _check(name, st)
    return out


def kv_attention(query, k_cache, v_cache, past_seq_lens, *, num_heads, scale=None, softcap=0.0, alibi_slopes=None,
                 document_ids=None, prefix_lens=None, out=None, status=None, workspace=None, stream=None):
    """Attention of the S newest tokens over the caches that the Q/K operators append to (see
    ``kv_attention`` in include/rope.h): query (B, S, num_heads*H) as rope_apply_qkv returns it, caches
    (B, kv_num_heads, max_len, H) after its append, past_seq_lens the lengths before it. scale: 1/sqrt(H)
    if None. workspace: uint8 device memory of ``kv_attention_workspace`` bytes, or None to take it from
    PyTorch's allocator for the call. Returns out."""
    return _attention("kv_attention", query, k_cache, v_cache, None, past_seq_lens, num_heads, scale, softcap,
                      alibi_slopes, document_ids, prefix_lens, out, status, workspace, stream)


def kv_attention_fp8(query, k_cache, v_cache, k_scale, v_scale, past_seq_lens, *, num_heads, scale=None, softcap=0.0,
                     alibi_slopes=None, document_ids=None, prefix_lens=None, out=None, status=None, workspace=None,
                     stream=None):
    """kv_attention over the 8-bit caches and scales of rope_apply_qkv_fp8."""
    return _attention("kv_attention_fp8", query, k_cache, v_cache, (k_scale, v_scale), past_seq_lens, num_heads,
                      scale, softcap, alibi_slopes, document_ids, prefix_lens, out, status, workspace, stream)


# --------------------------------------------------------------------------
# Caches held in pages
# --------------------------------------------------------------------------

def kv_cache_paged(num_pages, kv_num_heads, page_size, head_size, dtype=None, device=None):
    """Empty pages for rope_apply_qkv_paged: (k_pages, v_pages), each (num_pages, kv_num_heads, page_size,
    head_size)."""
    import torch

    shape = (num_pages, kv_num_heads, page_size, head_size)
    device = torch.device("cuda") if device is None else device
    return tuple(torch.zeros(shape, dtype=dtype or torch.float16, device=device) for _ in range(2))


def _paged(like, name, T, at, k_pages, v_pages, page_table, past_seq_lens, query_starts, i32):
    """(shape of the pages, elements between them, sequences, entries of a row of the table), checked together
    with the lengths; ``like``, the argument ``name``, says what device they have to be on."""
    plane, table = k_pages.shape, page_table.shape
    if not (at >= 0 and len(plane) == 4 and len(table) == 2 and k_pages.dtype is T and v_pages.dtype is T
            and page_table.dtype is i32 and past_seq_lens.dtype is i32 and v_pages.shape == plane
            and past_seq_lens.shape == table[:1] and k_pages.is_contiguous() and v_pages.is_contiguous()
            and page_table.is_contiguous() and past_seq_lens.is_contiguous() and k_pages.get_device() == at
            and v_pages.get_device() == at and page_table.get_device() == at and past_seq_lens.get_device() == at):
        if len(plane) != 4:
            raise ValueError("k_pages must be (num_pages, kv_num_heads, page_size, head_size)")
        if len(table) != 2:
            raise ValueError("page_table must be (B, max_pages)")
        if not like.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _shaped("page_table", page_table, like, table, i32)
        _shaped("past_seq_lens", past_seq_lens, like, table[:1], i32)
        for which, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.shape != plane or t.dtype != T or not t.is_cuda or t.device != like.device:
                raise ValueError(f"{which} must be a {T} tensor of shape {tuple(plane)} on {like.device}")
            if t.numel() and not t[0].is_contiguous():
                raise ValueError(f"{which} must be contiguous within a page")
        if plane[0] > 1 and k_pages.stride(0) != v_pages.stride(0):
            raise ValueError("k_pages and v_pages must have the same stride between pages")
    within = plane[1] * plane[2] * plane[3]
    stride = k_pages.stride(0) if plane[0] > 1 else within
    if stride < within:
        raise ValueError("pages must not overlap")
    if query_starts is not None and not (
            query_starts.dtype is i32 and query_starts.shape == (table[0] + 1,) and query_starts.is_contiguous()
            and query_starts.get_device() == at):
        _shaped("query_starts", query_starts, like, (table[0] + 1,), i32)
    return plane, stride, table[0], table[1]


def _tokens_of(query, query_starts, B):
    """(tokens, hidden) of query: (tokens, hidden) with query_starts, (B, S, hidden) without."""
    shape = query.shape
    if query_starts is None:
        if len(shape) != 3 or shape[0] != B:
            raise ValueError("query must be (B, S, hidden) with the batch of page_table, or come with query_starts")
        return B * shape[1], shape[2]
    if len(shape) != 2:
        raise ValueError("query must be (tokens, hidden) with query_starts")
    return shape


def rope_apply_qkv_paged(query, cos_cache, sin_cache, position_ids=None, *, num_heads, kv_num_heads, k_pages, v_pages,
                         page_table, past_seq_lens, query_starts=None, key=None, value=None, interleaved=0,
                         rotary_embedding_dim=0, q_out=None, status=None, q_norm_weight=None, k_norm_weight=None,
                         epsilon=1e-6, stream=None):
    """rope_apply_qkv in cache mode with caches held in pages (see ``rope_apply_qkv_paged`` in include/rope.h).

    query is (tokens, num_heads*H) with query_starts (int32 (B + 1)), or (B, S, num_heads*H) without, packed
    [Q|K|V] where key and value are None; position_ids has its leading dimensions. k_pages and v_pages
    (num_pages, kv_num_heads, page_size, H) are updated in place; they may be views of one tensor that holds K and V
    of each page side by side, for the other paged calls too. page_table is int32 (B, max_pages). Returns q_out."""
    T, at = query.dtype, query.get_device()
    torch, code = _torch_code(T)
    short = _short or _short_way()
    if short and stream is None and at >= 0 and at == torch._C._cuda_getDevice():
        done = short.append(at, torch._C._cuda_getCurrentRawStream(at), query, cos_cache, sin_cache, position_ids,
                            num_heads, kv_num_heads, k_pages, v_pages, page_table, past_seq_lens, query_starts, key, value,
                            interleaved, rotary_embedding_dim, q_out, status, q_norm_weight, k_norm_weight, epsilon)
        if done is not None:
            if done.__class__ is int:
                _check("rope_apply_qkv_paged", done)
            return done
    lib, dev = load_library(), query.device
    i32 = torch.int32
    (P, N, ps, H), stride, B, wide = _paged(query, "query", T, at, k_pages, v_pages, page_table, past_seq_lens, query_starts, i32)
    tokens, hidden = _tokens_of(query, query_starts, B)
    lead = query.shape[:-1]
    packed = key is None and value is None
    if N != kv_num_heads:
        raise ValueError(f"k_pages hold {N} heads, kv_num_heads is {kv_num_heads}")
    if hidden != (num_heads + (2 * kv_num_heads if packed else 0)) * H:
        raise ValueError(f"query hidden size {hidden} is not that of the heads of {H}")
    if cos_cache.dim() != 2:
        raise ValueError("cos_cache must be (rows, rd/2)")
    table = (cos_cache.shape[0], (rotary_embedding_dim or H) // 2)
    if not (query.is_contiguous() and _fits(cos_cache, at, table, T) and _fits(sin_cache, at, table, T)):
        _shaped("query", query, query, query.shape, T)
        _shaped("cos_cache", cos_cache, query, table, T)
        _shaped("sin_cache", sin_cache, query, table, T)
    if not packed:
        _shaped("key", key, query, (*lead, N * H), T)
        _shaped("value", value, query, (*lead, N * H), T)
    if q_norm_weight is not None or k_norm_weight is not None:
        _shaped("q_norm_weight", q_norm_weight, query, (H,), T)
        _shaped("k_norm_weight", k_norm_weight, query, (H,), T)
    if position_ids is not None:
        _shaped("position_ids", position_ids, query, lead, torch.int64)
    if q_out is not None:
        _shaped("q_out", q_out, query, (*lead, num_heads * H), T)
    if status is not None:
        _shaped("status", status, query, status.shape, i32)
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return rope_apply_qkv_paged(
                query, cos_cache, sin_cache, position_ids, num_heads=num_heads, kv_num_heads=kv_num_heads,
                k_pages=k_pages, v_pages=v_pages, page_table=page_table, past_seq_lens=past_seq_lens,
                query_starts=query_starts, key=key, value=value, interleaved=interleaved,
                rotary_embedding_dim=rotary_embedding_dim, q_out=q_out, status=status, q_norm_weight=q_norm_weight,
                k_norm_weight=k_norm_weight, epsilon=epsilon)
    if q_out is None:
        q_out = torch.empty((*lead, num_heads * H), dtype=T, device=dev)
    st = lib.rope_apply_qkv_paged(
        code, B, tokens, num_heads, N, H, query.data_ptr(), _address(key), _address(value), _address(q_norm_weight),
        _address(k_norm_weight), epsilon, cos_cache.data_ptr(), sin_cache.data_ptr(), table[0], _address(position_ids),
        past_seq_lens.data_ptr(), _address(query_starts), page_table.data_ptr(), wide, int(interleaved),
        rotary_embedding_dim, q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), P, ps, stride, _address(status),
        torch._C._cuda_getCurrentRawStream(at))
    if st:
        _check("rope_apply_qkv_paged", st)
    return q_out


def kv_attention_paged_workspace(dtype, batch, tokens, max_query_len, num_heads, kv_num_heads, head_size, page_size,
                                 max_pages):
    """Bytes of workspace that kv_attention_paged uses for such a call (max_query_len at most tokens here)."""
    n = load_library().kv_attention_paged_workspace(_torch_code(dtype)[1], batch, tokens, max_query_len, num_heads,
                                                    kv_num_heads, head_size, page_size, max_pages)
    if n < 0:
        _check("kv_attention_paged_workspace", ROPE_ERR_INVALID_ARG)
    return n


def kv_attention_paged(query, k_pages, v_pages, page_table, past_seq_lens, *, num_heads, query_starts=None,
                       max_query_len=None, scale=None, softcap=0.0, window=0, alibi_slopes=None, tree_masks=None,
                       out=None, status=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens over caches held in pages (see ``kv_attention_paged`` in
    include/rope.h), after rope_apply_qkv_paged with the same lengths and table.

    query is (tokens, num_heads*H) with query_starts (int32 (B + 1)), or (B, S, num_heads*H) without.
    max_query_len: at least the longest sequence's new tokens; None, or more than there are tokens: as many as
    there are, which plans worse (with more than 64 tokens tree_masks want it given). tree_masks: int64, one word a
    token, bit t: new token t of its sequence is seen. scale: 1/sqrt(H) if None. workspace: uint8 device memory of
    ``kv_attention_paged_workspace`` bytes, or None to take it from PyTorch's allocator. Returns out."""
    T, at = query.dtype, query.get_device()
    torch, code = _torch_code(T)
    short = _short or _short_way()
    if short and stream is None and at >= 0 and at == torch._C._cuda_getDevice():
        done = short.attention(at, torch._C._cuda_getCurrentRawStream(at), query, k_pages, v_pages, page_table,
                               past_seq_lens, num_heads, query_starts, max_query_len, scale, softcap, window, alibi_slopes,
                               tree_masks, out, status, workspace)
        if done is not None:
            if done.__class__ is int:
                _check("kv_attention_paged", done)
            return done
    lib, dev = load_library(), query.device
    i32 = torch.int32
    (P, N, ps, H), stride, B, wide = _paged(query, "query", T, at, k_pages, v_pages, page_table, past_seq_lens, query_starts, i32)
    tokens, hidden = _tokens_of(query, query_starts, B)
    if hidden != num_heads * H or not query.is_contiguous():
        _shaped("query", query, query, (*query.shape[:-1], num_heads * H), T)
    if max_query_len is None or query_starts is None:
        most = tokens if query_starts is not None else query.shape[1]
        if max_query_len not in (None, most):
            raise ValueError(f"max_query_len must be {most} without query_starts, got {max_query_len}")
        max_query_len = most
    max_query_len = min(max_query_len, tokens)
    if alibi_slopes is not None:
        _shaped("alibi_slopes", alibi_slopes, query, (num_heads,), torch.float32)
    if tree_masks is not None:
        _shaped("tree_masks", tree_masks, query, query.shape[:-1], torch.int64)
    if out is not None:
        _shaped("out", out, query, query.shape, T)
    if status is not None:
        _shaped("status", status, query, status.shape, i32)
    if workspace is not None:
        _shaped("workspace", workspace, query, workspace.shape, torch.uint8)
    if scale is None:
        scale = max(H, 1) ** -0.5
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return kv_attention_paged(query, k_pages, v_pages, page_table, past_seq_lens, num_heads=num_heads,
                                      query_starts=query_starts, max_query_len=max_query_len, scale=scale,
                                      softcap=softcap, window=window, alibi_slopes=alibi_slopes, tree_masks=tree_masks,
                                      out=out, status=status, workspace=workspace)
    if out is None:
        out = torch.empty_like(query)
    if workspace is None:
        need = _workspace(lib.kv_attention_paged_workspace, (code, B, tokens, max_query_len, num_heads, N, H, ps, wide))
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib.kv_attention_paged(
        code, B, tokens, max_query_len, num_heads, N, H, query.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), P, ps,
        stride, page_table.data_ptr(), wide, past_seq_lens.data_ptr(), _address(query_starts), scale, softcap, window,
        _address(alibi_slopes), _address(tree_masks), out.data_ptr(), _address(status), _address(workspace),
        0 if workspace is None else workspace.numel(), torch._C._cuda_getCurrentRawStream(at))
    if st:
        _check("kv_attention_paged", st)
    return out


def kv_keep_paged(k_pages, v_pages, page_table, past_seq_lens, kept, kept_lens, *, status=None, stream=None):
    """After drafts were verified: row past_seq_lens[b] + kept[b, i] of each sequence goes to past_seq_lens[b] + i
    for i < kept_lens[b], in k_pages and v_pages (see ``kv_keep_paged`` in include/rope.h). kept is int32 (B,
    max_kept), ascending; kept_lens int32 (B). The next past_seq_lens is past_seq_lens + kept_lens."""
    T, at = k_pages.dtype, k_pages.get_device()
    torch, code = _torch_code(T)
    short = _short or _short_way()
    if short and stream is None and at >= 0 and at == torch._C._cuda_getDevice():
        done = short.keep(at, torch._C._cuda_getCurrentRawStream(at), k_pages, v_pages, page_table, past_seq_lens, kept,
                          kept_lens, status)
        if done is not None:
            if done.__class__ is int:
                _check("kv_keep_paged", done)
            return
    lib, dev = load_library(), k_pages.device
    i32 = torch.int32
    (P, N, ps, H), stride, B, wide = _paged(k_pages, "k_pages", T, at, k_pages, v_pages, page_table, past_seq_lens, None, i32)
    if kept.dim() != 2:
        raise ValueError("kept must be (B, max_kept)")
    most = kept.shape[1]
    if not (_fits(kept, at, (B, most), i32) and _fits(kept_lens, at, (B,), i32)):
        _shaped("kept", kept, k_pages, (B, most), i32)
        _shaped("kept_lens", kept_lens, k_pages, (B,), i32)
    if status is not None:
        _shaped("status", status, k_pages, status.shape, i32)
    if _elsewhere(torch, dev, stream):
        with _on(dev, stream):
            return kv_keep_paged(k_pages, v_pages, page_table, past_seq_lens, kept, kept_lens, status=status)
    st = lib.kv_keep_paged(
        code, B, N, H, k_pages.data_ptr(), v_pages.data_ptr(), P, ps, stride, page_table.data_ptr(), wide,
        past_seq_lens.data_ptr(), kept.data_ptr(), most, kept_lens.data_ptr(), _address(status),
        torch._C._cuda_getCurrentRawStream(at))
    if st:
        _check("kv_keep_paged", st)


def set_variant(name):
    """Kernel variant for later calls in this process: "auto", "simt" or "tma"."""
    lib = load_library()
    _check("rope_set_variant", lib.rope_set_variant(VARIANTS[name]))
    _workspace_bytes.clear()


def get_variant():
    code = load_library().rope_get_variant()
    return {v: k for k, v in VARIANTS.items()}[code]


def last_kernel():
    """Kernel family the calling thread's last launching call used ("" before any)."""
    return load_library().rope_last_kernel().decode()


class variant:
    """Context manager: ``with variant("tma"): ...``."""

    def __init__(self, name):
        self.name = name

    def __enter__(self):
        self.prev = get_variant()
        set_variant(self.name)
        return self

    def __exit__(self, *exc):
        set_variant(self.prev)
