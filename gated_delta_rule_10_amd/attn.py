"""Python binding of libkda's attention entry points (include/kda_attn.h):
argument marshalling only, as gated_delta_rule_10_amd.kda is for the KDA
operator. Every step runs in the HIP kernels of libkda.so; if the library is
not built, or a tensor is not on a GPU, the functions raise.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import kda
from .kda import KDA_ERR_WORKSPACE, KDA_OK, KDAError, _code, _dev, _one_device, _out, _ptr, _stream

KDA_KV_F32, KDA_KV_BF16, KDA_KV_E4M3 = range(3)
_KV_CODES = {torch.float32: KDA_KV_F32, torch.bfloat16: KDA_KV_BF16, torch.float8_e4m3fn: KDA_KV_E4M3}


class KdaKvCache(ctypes.Structure):
    """kda_kv_cache_t of include/kda_attn.h (field order and C types as declared there)."""
    _fields_ = [("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p),
                ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32),
                ("dtype", ctypes.c_int)]


_lib = None


def load_library() -> ctypes.CDLL:
    """libkda.so with the attention entry points' C signatures (no HIP call is made)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = kda.load_library()
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    cache = ctypes.POINTER(KdaKvCache)
    lib.kda_attn_fwd.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, i32, i64, i64, i64, ctypes.c_int, ctypes.c_int,
                                 f32, P, P]
    lib.kda_kv_write.argtypes = [P, P, P, i32, i32, i32, i32, i32, i64, i64, ctypes.c_int, cache, P]
    lib.kda_kv_read.argtypes = [P, P, P, i32, i32, i32, i32, i32, ctypes.c_int, cache, P]
    lib.kda_attn_cache_fwd.argtypes = [P, P, i32, i32, i32, i32, i32, i32, i64, ctypes.c_int, ctypes.c_int, f32, cache,
                                       P, P, P, sz, P]
    for f in (lib.kda_attn_fwd, lib.kda_kv_write, lib.kda_kv_read, lib.kda_attn_cache_fwd):
        f.restype = ctypes.c_int
    lib.kda_attn_cache_fwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, ctypes.c_int]
    lib.kda_attn_cache_fwd_workspace_size.restype = sz
    _lib = lib
    return lib


def _rows(t: torch.Tensor, name: str) -> int:
    """Token stride, in elements, of a [T, heads, d] GPU tensor whose [heads, d] part is dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, d]")
    T, h, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads and channels of a token must be contiguous")
    return st if T > 1 else h * d


def _dense(device, **tensors) -> None:
    """Every tensor given (None skipped) contiguous and on `device`, a GPU: the call runs there."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device != device or not t.is_contiguous():
            _dev(t, name)
            _one_device(device, t)


def _offsets(cu_seqlens: torch.Tensor) -> int:
    """N of a cu_seqlens tensor."""
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be int32 [N + 1]")
    return cu_seqlens.shape[0] - 1


def _cache(device, N: int, cache_lens, page_table, k_cache, v_cache, k_exp, v_exp) -> KdaKvCache:
    """The call's cache, after checking its tensors against each other."""
    _dense(device, cache_lens=cache_lens, page_table=page_table, k_cache=k_cache, v_cache=v_cache, k_exp=k_exp, v_exp=v_exp)
    if cache_lens.dtype != torch.int32 or cache_lens.shape != (N,):
        raise ValueError("cache_lens must be int32 [N]")
    rows = page_table.shape
    if page_table.dtype != torch.int32 or len(rows) != 2 or rows[0] != N:
        raise ValueError("page_table must be int32 [N, max_pages]")
    kind, shape, vshape = k_cache.dtype, k_cache.shape, v_cache.shape
    if len(shape) != 4 or len(vshape) != 4 or shape[:3] != vshape[:3] or v_cache.dtype != kind:
        raise ValueError("k_cache and v_cache must be [num_pages, Hk, page_size, d] of one dtype")
    code = _KV_CODES.get(kind)
    if code is None:
        raise TypeError(f"unsupported cache dtype {kind}")
    ke = ve = None
    if code == KDA_KV_E4M3:
        if k_exp is None or v_exp is None:
            raise ValueError("an e4m3 cache needs k_exp and v_exp")
        if k_exp.dtype != torch.uint8 or v_exp.dtype != torch.uint8 or not k_exp.shape == v_exp.shape == shape[:3]:
            raise ValueError("k_exp and v_exp must be uint8 [num_pages, Hk, page_size]")
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    elif k_exp is not None or v_exp is not None:
        raise ValueError("k_exp and v_exp are for e4m3 caches")
    return KdaKvCache(k_cache.data_ptr(), v_cache.data_ptr(), ke, ve, page_table.data_ptr(), cache_lens.data_ptr(),
                      shape[0], shape[2], rows[1], code)


class _Here:
    """A context that changes nothing."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device):
    """The device as the current one (entering torch.cuda.device costs more than asking)."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _handle(stream, device) -> int:
    """The stream to enqueue on, as its handle: the given one (of `device`), else the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return _stream(stream, device).value or 0


def _alloc_on(stream):
    """New tensors of a call come from the pool of the stream that the call runs on."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def kda_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                 scale: Optional[float] = None, out_dtype: Optional[torch.dtype] = None,
                 o: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention inside packed sequences (kda_attn_fwd of include/kda_attn.h).

    q: [T, H, d_k]; k: [T, Hk, d_k]; v: [T, Hk, d_v], bf16 or fp32, H a multiple of Hk, each with a token
    stride of its own; cu_seqlens: int32 [N + 1]; scale: 1 / sqrt(d_k) if None. Returns o [T, H, d_v]
    (rows from cu_seqlens[N] on are left as they were).
    """
    lib = load_library()
    sq, sk, sv = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    N = _offsets(cu_seqlens)
    T, H, d_k = q.shape
    Hk, d_v = v.shape[1], v.shape[2]
    if k.shape != (T, Hk, d_k) or v.shape[0] != T or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("inconsistent q/k/v shapes or dtypes")
    out_dtype = q.dtype if out_dtype is None else out_dtype
    device = q.device
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            o = _out(o, (T, H, d_v), out_dtype, device)
        _dense(device, cu_seqlens=cu_seqlens, o=o)
        _one_device(device, k, v)
        st = lib.kda_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), N, T, H, Hk, d_k, d_v,
                              sq, sk, sv, _code(q.dtype), _code(out_dtype),
                              d_k ** -0.5 if scale is None else float(scale), o.data_ptr(), s)
    if st != KDA_OK:
        raise KDAError(st, "kda_attn_fwd")
    return o


def kda_kv_write(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor,
                 page_table: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, *,
                 k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None, stream=None) -> None:
    """New tokens into the paged cache (kda_kv_write of include/kda_attn.h).

    k: [T, Hk, d_k]; v: [T, Hk, d_v]; cu_seqlens: int32 [N + 1] of the new tokens; cache_lens: int32 [N], the
    tokens of each sequence in the cache with the new ones; page_table: int32 [N, max_pages]; k_cache, v_cache:
    [num_pages, Hk, page_size, d], fp32 (fp32 inputs), bf16 or float8_e4m3fn (bf16 inputs), the latter with
    k_exp, v_exp: uint8 [num_pages, Hk, page_size].
    """
    lib = load_library()
    sk, sv = _rows(k, "k"), _rows(v, "v")
    N = _offsets(cu_seqlens)
    T, Hk, d_k = k.shape
    d_v = v.shape[2]
    if v.shape[:2] != (T, Hk) or k.dtype != v.dtype:
        raise ValueError("inconsistent k/v shapes or dtypes")
    device = k.device
    _dense(device, cu_seqlens=cu_seqlens)
    _one_device(device, v)
    cache = _cache(device, N, cache_lens, page_table, k_cache, v_cache, k_exp, v_exp)
    if k_cache.shape[1] != Hk or k_cache.shape[3] != d_k or v_cache.shape[3] != d_v:
        raise ValueError("k_cache and v_cache must have the heads and channels of k and v")
    with _on(device):
        st = lib.kda_kv_write(k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), N, T, Hk, d_k, d_v, sk, sv,
                              _code(k.dtype), ctypes.byref(cache), _handle(stream, device))
    if st != KDA_OK:
        raise KDAError(st, "kda_kv_write")


def kda_kv_read(T: int, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor, page_table: torch.Tensor,
                k_cache: torch.Tensor, v_cache: torch.Tensor, *, k_exp: Optional[torch.Tensor] = None,
                v_exp: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The last cu_seqlens[n + 1] - cu_seqlens[n] cached tokens of every sequence (kda_kv_read of
    include/kda_attn.h; the cache's arguments as for kda_kv_write), T = cu_seqlens[N] of them in all.
    Returns (k [T, Hk, d_k], v [T, Hk, d_v]) of out_dtype.
    """
    lib = load_library()
    N = _offsets(cu_seqlens)
    device = k_cache.device
    _dense(device, cu_seqlens=cu_seqlens)
    cache = _cache(device, N, cache_lens, page_table, k_cache, v_cache, k_exp, v_exp)
    Hk, d_k, d_v = k_cache.shape[1], k_cache.shape[3], v_cache.shape[3]
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            k = _out(k, (T, Hk, d_k), out_dtype, device)
            v = _out(v, (T, Hk, d_v), out_dtype, device)
        _dense(device, k=k, v=v)
        st = lib.kda_kv_read(k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), N, T, Hk, d_k, d_v, _code(out_dtype),
                             ctypes.byref(cache), s)
    if st != KDA_OK:
        raise KDAError(st, "kda_kv_read")
    return k, v


def kda_attn_cache_fwd_workspace_size(N: int, T: int, H: int, Hk: int, d_k: int, d_v: int, max_tokens: int,
                                      in_dtype: torch.dtype) -> int:
    """Bytes on the current device; max_tokens: what the page table reaches, max_pages * page_size."""
    return int(load_library().kda_attn_cache_fwd_workspace_size(N, T, H, Hk, d_k, d_v, max_tokens, _code(in_dtype)))


def kda_attn_cache_fwd(q: torch.Tensor, cu_seqlens: torch.Tensor, cache_lens: torch.Tensor, page_table: torch.Tensor,
                       k_cache: torch.Tensor, v_cache: torch.Tensor, *, k_exp: Optional[torch.Tensor] = None,
                       v_exp: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, out_dtype: Optional[torch.dtype] = None,
                       o: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Attention of new tokens over the cache that holds them already (kda_attn_cache_fwd of
    include/kda_attn.h; the cache's arguments as for kda_kv_write).

    q: [T, H, d_k], with a token stride of its own; cu_seqlens: int32 [N + 1] of the new tokens; tree_mask:
    int64 [T] or None: bit b of a token's word lets it see new token b of its sequence (None: those up to and
    including itself); scale: 1 / sqrt(d_k) if None. Returns o [T, H, d_v] (rows from cu_seqlens[N] on are left
    as they were).
    """
    lib = load_library()
    sq = _rows(q, "q")
    N = _offsets(cu_seqlens)
    T, H, d_k = q.shape
    device = q.device
    _dense(device, cu_seqlens=cu_seqlens, tree_mask=tree_mask)
    cache = _cache(device, N, cache_lens, page_table, k_cache, v_cache, k_exp, v_exp)
    Hk, d_v = k_cache.shape[1], v_cache.shape[3]
    if k_cache.shape[3] != d_k:
        raise ValueError("q and k_cache must have the same channels")
    if tree_mask is not None and (tree_mask.dtype != torch.int64 or tree_mask.shape != (T,)):
        raise ValueError("tree_mask must be int64 [T]")
    out_dtype = q.dtype if out_dtype is None else out_dtype
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            o = _out(o, (T, H, d_v), out_dtype, device)
            if workspace is None:
                need = lib.kda_attn_cache_fwd_workspace_size(N, T, H, Hk, d_k, d_v, cache.max_pages * cache.page_size,
                                                             _code(q.dtype))
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=device)
        _dense(device, o=o, workspace=workspace)
        st = lib.kda_attn_cache_fwd(q.data_ptr(), cu_seqlens.data_ptr(), N, T, H, Hk, d_k, d_v, sq, _code(q.dtype),
                                    _code(out_dtype), d_k ** -0.5 if scale is None else float(scale),
                                    ctypes.byref(cache), _ptr(tree_mask), o.data_ptr(), _ptr(workspace),
                                    0 if workspace is None else workspace.numel() * workspace.element_size(), s)
    if st != KDA_OK:
        where = "kda_attn_cache_fwd"
        if st == KDA_ERR_WORKSPACE:
            where += " (kda_attn_cache_fwd_workspace_size)"
        raise KDAError(st, where)
    return o
