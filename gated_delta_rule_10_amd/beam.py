"""Python binding of libkda's beam-search entry points (include/kda_beam.h):
argument marshalling only. Every step runs in the HIP kernels of libkda.so; if
the library is not built, or a tensor is not on a GPU, the functions raise.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import kda
from .attn import _alloc_on, _dense, _handle, _on
from .kda import KDA_ERR_WORKSPACE, KDA_OK, KDAError, _code, _out, _ptr

_lib = None


def load_library() -> ctypes.CDLL:
    """libkda.so with the beam-search entry points' C signatures (no HIP call is made)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = kda.load_library()
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kda_beam_select.argtypes = [P, i64, P, P, i32, i32, i32, i32, i32, ctypes.c_int, P, P, P, P, sz, P]
    lib.kda_state_reorder.argtypes = [P, i64, i32, i32, i64, P, P, P, i32, i32, P]
    lib.kda_beam_select.restype = lib.kda_state_reorder.restype = ctypes.c_int
    lib.kda_beam_select_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.kda_beam_select_workspace_size.restype = sz
    _lib = lib
    return lib


def kda_beam_select_workspace_size(N: int, W: int, V: int, K: int) -> int:
    """Bytes on the current device."""
    return int(load_library().kda_beam_select_workspace_size(N, W, V, K))


def kda_beam_select(logits: torch.Tensor, scores: torch.Tensor, K: int, *, done: Optional[torch.Tensor] = None,
                    done_token: int = 0, out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The K best (beam, token) pairs of every request (kda_beam_select of include/kda_beam.h).

    logits: [N, W, V], bf16 or fp32, rows of V contiguous, the rows themselves evenly apart; scores: fp32
    [N, W]; done: uint8 or bool [N, W] or None, beams that have ended and keep their score with done_token.
    Returns (scores fp32, parent int32, token int32), each [N, K] (or the caller's three tensors `out`).
    """
    lib = load_library()
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    if logits.dim() != 3:
        raise ValueError("logits must be [N, W, V]")
    N, W, V = logits.shape
    sn, sw, sv = logits.stride()
    row = sw if W > 1 else sn if N > 1 else V
    if (sv != 1 and V > 1) or (N > 1 and sn != W * row):
        raise ValueError("logits: rows must be contiguous and evenly apart")
    device = logits.device
    if scores.dtype != torch.float32 or scores.shape != (N, W):
        raise ValueError("scores must be float32 [N, W]")
    if done is not None and (done.dtype not in (torch.uint8, torch.bool) or done.shape != (N, W)):
        raise ValueError("done must be uint8 or bool [N, W]")
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            best, parent, token = out or (None, None, None)
            best = _out(best, (N, K), torch.float32, device)
            parent = _out(parent, (N, K), torch.int32, device)
            token = _out(token, (N, K), torch.int32, device)
            if workspace is None:
                need = lib.kda_beam_select_workspace_size(N, W, V, K)
                if need:
                    workspace = torch.empty(need, dtype=torch.uint8, device=device)
        _dense(device, scores=scores, done=done, best=best, parent=parent, token=token, workspace=workspace)
        st = lib.kda_beam_select(logits.data_ptr(), row, scores.data_ptr(), _ptr(done), int(done_token), N, W, V, K,
                                 _code(logits.dtype), best.data_ptr(), parent.data_ptr(), token.data_ptr(), _ptr(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(), s)
    if st != KDA_OK:
        where = "kda_beam_select"
        if st == KDA_ERR_WORKSPACE:
            where += " (kda_beam_select_workspace_size)"
        raise KDAError(st, where)
    return best, parent, token


def kda_state_reorder(states: torch.Tensor, slots: torch.Tensor, parent: torch.Tensor, *,
                      slots_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """States and slots after a choice of parents (kda_state_reorder of include/kda_beam.h).

    states: [layers, num_slots, ...] of any dtype, a layer's part contiguous, updated in place (a cache of one
    layer: cache[None]); slots, parent: int32 [N, W]. Returns the beams' slots afterwards, int32 [N, W].
    """
    lib = load_library()
    if not states.is_cuda:
        raise ValueError("states must be a GPU tensor")
    if states.dim() < 3:
        raise ValueError("states must be [layers, num_slots, ...]")
    layers, num_slots = states.shape[:2]
    row = 1  # elements: of a slot's row in the end
    for i, (n, stride) in enumerate(zip(states.shape[:0:-1], states.stride()[:0:-1])):
        if n > 1 and stride != row:
            raise ValueError("states: every layer's part must be contiguous")
        if i < states.dim() - 2:
            row *= n
    size = states.element_size()
    device = states.device
    for name, t in (("slots", slots), ("parent", parent)):
        if t.dtype != torch.int32 or t.dim() != 2 or t.shape != slots.shape:
            raise ValueError(f"{name} must be int32 [N, W]")
    N, W = slots.shape
    with _on(device):
        s = _handle(stream, device)
        with _alloc_on(stream):
            slots_out = _out(slots_out, (N, W), torch.int32, device)
        _dense(device, slots=slots, parent=parent, slots_out=slots_out)
        st = lib.kda_state_reorder(states.data_ptr(), states.stride(0) * size, layers, num_slots, row * size, slots.data_ptr(),
                                   parent.data_ptr(), slots_out.data_ptr(), N, W, s)
    if st != KDA_OK:
        raise KDAError(st, "kda_state_reorder")
    return slots_out
