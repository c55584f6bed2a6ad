"""Python binding of include/kda_linear.h: linear attention with a decay per head.

    S <- a S + k v^T ;  o = S^T q      (a scalar decay per head)

on the slot cache of kda_decode_step. As in kda.py, each function has the name
of its C entry point, takes torch tensors that live on the GPU and raises
KdaError on a non-zero status. The kernels go to the current stream of the
tensors' device, or to ``stream``, whichever device is current.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .kda import KDA_OK, KdaError, load_library
from .native import native


class kda_lin_tokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("alpha_stride", ctypes.c_int64), ("Hk", ctypes.c_int32)]


def kda_lin_decode_step(cache: torch.Tensor, slot_ids: torch.Tensor, q, k, v, alpha, out: torch.Tensor, *,
                        gate=None, weight=None, eps: float = 1e-6, dev_err: Optional[torch.Tensor] = None,
                        tile_w: int = 0, stream=None) -> None:
    """One token per row, state updated in place.

    cache float32 [num_slots, H, dv, dk]; slot_ids int32 [B]; q, k bf16 [B, Hk, dk] with Hk dividing
    H; v bf16 [B, H, dv]; alpha float32 [H] (fixed) or [B, H] (q, k, v and alpha may be slices with any
    stride between tokens); out float32 or bf16 [B, H, dv], 16-byte aligned (bf16: 8); gate bf16
    [B, H, dv] (optional output gate), 8-byte aligned; weight float32 [dv].
    """
    rc = native().lin_decode_step(cache, slot_ids, q, k, v, alpha, out, gate, weight, eps, dev_err, tile_w, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_lin_decode_step")


def kda_lin_prefill_workspace(B: int, n_tok: int, H: int, dk: int, dv: int) -> int:
    """Workspace bytes kda_lin_prefill needs for these sizes (0: none), never less for a larger B or n_tok."""
    n = ctypes.c_size_t(0)
    rc = load_library().kda_lin_prefill_workspace(B, n_tok, H, dk, dv, ctypes.byref(n))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_lin_prefill_workspace")
    return n.value


def kda_lin_prefill(cache: torch.Tensor, slot_ids: torch.Tensor, cu_seqlens: torch.Tensor, q, k, v, alpha,
                    out: torch.Tensor, *, ckpt_pos: Optional[torch.Tensor] = None,
                    ckpt: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Whole prompts with an optional in-pass checkpoint. Token arrays are as for kda_lin_decode_step
    with n_tok tokens; row b owns tokens [cu_seqlens[b], cu_seqlens[b + 1]); ckpt_pos int32 [B], ckpt
    float32 [B, H, dv, dk]. workspace: a contiguous tensor of any dtype, at least
    kda_lin_prefill_workspace() bytes; None allocates one for the call, on the stream that it runs on."""
    rc = native().lin_prefill(cache, slot_ids, cu_seqlens, q, k, v, alpha, out, ckpt_pos, ckpt, workspace, dev_err,
                              stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_lin_prefill")
