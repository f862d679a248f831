"""Python binding of libkda's linear-attention entry points (include/kda_lin.h):
argument marshalling only, as gated_delta_rule_10_amd.kda is for the KDA
operator. Every step runs in the HIP kernels of libkda.so; if the library is
not built, or a tensor is not on a GPU, the functions raise.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import kda
from .attn import _alloc_on, _dense, _handle, _offsets, _on, _rows
from .kda import KDA_ERR_WORKSPACE, KDA_OK, KDAError, _code, _one_device, _out, _ptr

_lib = None


def load_library() -> ctypes.CDLL:
    """libkda.so with the linear-attention entry points' C signatures (no HIP call is made)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = kda.load_library()
    P, i32, i64, f32, sz, en = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t,
                                ctypes.c_int)
    lib.kda_lin_chunk_fwd.argtypes = [P, P, P, P, P, i32, i32, i32, i32, i32, i32, i64, i64, i64, i64, en, en, f32, P, P, P,
                                      i32, P, P, sz, P]
    lib.kda_lin_decode_step.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i64, i64, i64, i64, i32, en, en, f32, P]
    lib.kda_lin_chunk_fwd.restype = lib.kda_lin_decode_step.restype = en
    lib.kda_lin_chunk_fwd_workspace_size.argtypes = [i32, i32, i32, i32, i32, en]
    lib.kda_lin_chunk_fwd_workspace_size.restype = sz
    _lib = lib
    return lib


def _tokens(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> Tuple[int, int, int]:
    """Token strides of [T, heads, d] GPU tensors; any strides will do where there is no token."""
    if v.dim() == 3 and v.shape[0] == 0:
        q, k, v = (t.new_empty((0,) + t.shape[1:]) if t.dim() == 3 and t.shape[0] == 0 else t for t in (q, k, v))
    return _rows(q, "q"), _rows(k, "k"), _rows(v, "v")


def _decay(g: torch.Tensor, T: int, H: int, device) -> int:
    """Token stride of log_decay: [T, H] with a token stride of its own, or [H] (0)."""
    if g.dtype != torch.float32:
        raise ValueError("log_decay must be float32")
    if g.device != device:
        raise ValueError(f"log_decay must be on {device}")
    if g.shape == (H,):
        if g.stride(0) != 1 and H > 1:
            raise ValueError("log_decay: the heads must be contiguous")
        return 0
    if g.shape != (T, H):
        raise ValueError("log_decay must be [T, H] or [H]")
    if T == 0:
        return H
    if g.stride(1) != 1 and H > 1:
        raise ValueError("log_decay: the heads of a token must be contiguous")
    return g.stride(0) if T > 1 else H


def _heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> None:
    dtype, shape = q.dtype, q.shape
    if k.shape != shape or v.shape[0] != shape[0] or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("inconsistent q/k/v shapes or dtypes")


def kda_lin_chunk_fwd_workspace_size(N: int, T: int, H: int, d_k: int, d_v: int, in_dtype: torch.dtype) -> int:
    """Bytes on the current device."""
    return int(load_library().kda_lin_chunk_fwd_workspace_size(N, T, H, d_k, d_v, _code(in_dtype)))


def kda_lin_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                      cu_seqlens: torch.Tensor, *, scale: float = 1.0, initial_state: Optional[torch.Tensor] = None,
                      output_final_state: bool = True, final_state: Optional[torch.Tensor] = None,
                      state_slots: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      o: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with one decay per head over packed sequences (kda_lin_chunk_fwd of include/kda_lin.h).

    q, k: [T, Hk, d_k]; v: [T, H, d_v], bf16 or fp32, H a multiple of Hk, each with a token stride of its own;
    log_decay: fp32 [T, H], or [H] for all tokens; cu_seqlens: int32 [N + 1]; initial_state: fp32
    [N, H, d_k, d_v] or None. With state_slots (int32 [N]), initial_state is a cache [slots, H, d_k, d_v] and
    final_state defaults to that same cache (updated in place). Returns (o [T, H, d_v], final_state).
    """
    lib = load_library()
    sq, sk, sv = _tokens(q, k, v)
    N = _offsets(cu_seqlens)
    _heads(q, k, v)
    T, Hk, d_k = q.shape
    H, d_v = v.shape[1], v.shape[2]
    device = q.device
    sg = _decay(log_decay, T, H, device)
    out_dtype = q.dtype if out_dtype is None else out_dtype
    slots = N
    if state_slots is not None:
        if state_slots.dtype != torch.int32 or state_slots.shape != (N,):
            raise ValueError("state_slots must be int32 [N]")
        if initial_state is None:
            raise ValueError("state_slots needs the state cache as initial_state")
        slots = initial_state.shape[0]
        if final_state is None and output_final_state:
            final_state = initial_state
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (slots, H, d_k, d_v)):
            raise ValueError(f"{name} must be float32 [{'N' if state_slots is None else 'slots'}, H, d_k, d_v]")
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            o = _out(o, (T, H, d_v), out_dtype, device)
            if final_state is None and output_final_state:
                final_state = torch.empty((N, H, d_k, d_v), dtype=torch.float32, device=device)
            if workspace is None:
                need = lib.kda_lin_chunk_fwd_workspace_size(N, T, H, d_k, d_v, _code(q.dtype))
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=device)
        _dense(device, cu_seqlens=cu_seqlens, initial_state=initial_state, final_state=final_state,
               state_slots=state_slots, o=o, workspace=workspace)
        _one_device(device, k, v)
        st = lib.kda_lin_chunk_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), cu_seqlens.data_ptr(),
                                   N, T, H, Hk, d_k, d_v, sq, sk, sv, sg, _code(q.dtype), _code(out_dtype), float(scale),
                                   _ptr(initial_state), _ptr(final_state), _ptr(state_slots), slots, o.data_ptr(),
                                   _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), s)
    if st != KDA_OK:
        where = "kda_lin_chunk_fwd"
        if st == KDA_ERR_WORKSPACE:
            where += " (kda_lin_chunk_fwd_workspace_size)"
        raise KDAError(st, where)
    return o, final_state


def kda_lin_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                        state_cache: torch.Tensor, slot_idx: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                        out_dtype: Optional[torch.dtype] = None, o: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """One token per sequence (kda_lin_decode_step of include/kda_lin.h), updating state_cache
    [slots, H, d_k, d_v] fp32 in place.

    q, k: [B, Hk, d_k]; v: [B, H, d_v], each with a token stride of its own; log_decay: fp32 [B, H] or [H];
    slot_idx: int32 [B] or None. Returns o [B, H, d_v].
    """
    lib = load_library()
    sq, sk, sv = _tokens(q, k, v)
    _heads(q, k, v)
    B, Hk, d_k = q.shape
    H, d_v = v.shape[1], v.shape[2]
    device = q.device
    sg = _decay(log_decay, B, H, device)
    if state_cache.dtype != torch.float32 or state_cache.dim() != 4 or state_cache.shape[1:] != (H, d_k, d_v):
        raise ValueError("state_cache must be float32 [slots, H, d_k, d_v]")
    if slot_idx is not None and (slot_idx.dtype != torch.int32 or slot_idx.shape != (B,)):
        raise ValueError("slot_idx must be int32 [B]")
    out_dtype = q.dtype if out_dtype is None else out_dtype
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            o = _out(o, (B, H, d_v), out_dtype, device)
        _dense(device, state_cache=state_cache, slot_idx=slot_idx, o=o)
        _one_device(device, k, v)
        st = lib.kda_lin_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state_cache.data_ptr(),
                                     _ptr(slot_idx), o.data_ptr(), B, H, Hk, d_k, d_v, sq, sk, sv, sg,
                                     state_cache.shape[0], _code(q.dtype), _code(out_dtype), float(scale), s)
    if st != KDA_OK:
        raise KDAError(st, "kda_lin_decode_step")
    return o
