"""Python binding of include/kda_linear.h: linear attention with a decay per head.

    S <- a S + k v^T ;  o = S^T q      (a scalar decay per head)

on the slot cache of kda_decode_step. As in kda.py, each function has the name
of its C entry point, takes torch tensors that live on the GPU and raises
KdaError on a non-zero status. The kernels go to the current stream of the
tensors' device, or to ``stream``, whichever device is current.
"""

from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from .kda import _BF16_TYPES, KDA_OK, KDA_OUT_BF16, KdaError, kda_epilogue, kda_options, load_library


class kda_lin_tokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("alpha_stride", ctypes.c_int64), ("Hk", ctypes.c_int32)]


# The same layout, packed at a third of the cost of the ctypes structure: a small
# call is bound by this binding, not by its kernel.
_TOKENS = struct.Struct("@QQQQqqqqi4x")
assert _TOKENS.size == ctypes.sizeof(kda_lin_tokens)

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_OUT = (torch.float32,) + _BF16_TYPES


def _refuse(dev: int, t, name: str, dtypes, shape) -> None:
    """Why tensor t is not one of the given types and shape on GPU ``dev``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on(dev: int, t, name: str, dtypes, shape) -> int:
    """Address of a contiguous tensor of the given types and shape on GPU ``dev``."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev and t.shape == shape):
        _refuse(dev, t, name, dtypes, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(dev: int, t, name: str, rows: int, heads: int, d: int):
    """(address, stride between tokens) of a bf16 [rows, heads, d] tensor whose heads are contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype in _BF16_TYPES and t.get_device() == dev
            and t.shape == (rows, heads, d)):
        _refuse(dev, t, name, _BF16_TYPES, (rows, heads, d))
    s = t.stride()
    if s[2] != 1 or (s[1] != d and heads > 1):
        raise ValueError(f"{name}: each token's heads must be contiguous, got strides {s}")
    return t.data_ptr(), (s[0] if rows > 1 else heads * d)


def _tokens(dev: int, rows: int, H: int, dk: int, dv: int, q, k, v, alpha) -> bytes:
    """The kda_lin_tokens of a call."""
    Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    if Hk < 1 or H % Hk:
        raise ValueError(f"k must be [rows, Hk, dk] with Hk dividing H = {H}")
    qp, qs = _heads(dev, q, "q", rows, Hk, dk)
    kp, ks = _heads(dev, k, "k", rows, Hk, dk)
    vp, vs = _heads(dev, v, "v", rows, H, dv)
    if isinstance(alpha, torch.Tensor) and alpha.dim() == 1:
        return _TOKENS.pack(qp, kp, vp, _on(dev, alpha, "alpha", _F32, (H,)), qs, ks, vs, 0, Hk)
    return _TOKENS.pack(qp, kp, vp, _on(dev, alpha, "alpha", _F32, (rows, H)), qs, ks, vs, H, Hk)


def _cache(cache):
    """cache: float32 [num_slots, H, dv, dk]; each slot contiguous, slots at stride(0)."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda or cache.dtype is not torch.float32 or cache.dim() != 4:
        raise ValueError("cache must be a float32 GPU tensor [num_slots, H, dv, dk]")
    ns, H, dv, dk = cache.shape
    s = cache.stride()
    if s[1:] != (dv * dk, dk, 1):
        raise ValueError("each cache slot must be contiguous [H, dv, dk]")
    return cache.get_device(), ns, (s[0] if ns > 1 else H * dv * dk), H, dv, dk


def _call(dev: int, fn, name: str, *args) -> None:
    """The entry point, with the tensors' device current."""
    if torch.cuda.current_device() == dev:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != KDA_OK:
        raise KdaError(rc, name)


# The current stream's handle without building a Stream object, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream_of(dev: int, stream) -> int:
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_BF16_OUT = kda_options(0, 0, KDA_OUT_BF16)


def _options(tile_w: int, out: torch.Tensor):
    bf16 = out.dtype is not torch.float32
    if tile_w:
        return ctypes.byref(kda_options(int(tile_w), 0, KDA_OUT_BF16 if bf16 else 0))
    return ctypes.byref(_BF16_OUT) if bf16 else None


def kda_lin_decode_step(cache: torch.Tensor, slot_ids: torch.Tensor, q, k, v, alpha, out: torch.Tensor, *,
                        gate=None, weight=None, eps: float = 1e-6, dev_err: Optional[torch.Tensor] = None,
                        tile_w: int = 0, stream=None) -> None:
    """One token per row, state updated in place.

    cache float32 [num_slots, H, dv, dk]; slot_ids int32 [B]; q, k bf16 [B, Hk, dk] with Hk dividing
    H; v bf16 [B, H, dv] (q, k, v may be slices with any stride between tokens); alpha float32 [H]
    (fixed) or [B, H]; out float32 or bf16 [B, H, dv]; gate bf16 [B, H, dv] (optional output gate),
    weight float32 [dv].
    """
    dev, ns, stride, H, dv, dk = _cache(cache)
    B = slot_ids.shape[0]
    slots = _on(dev, slot_ids, "slot_ids", _I32, (B,))
    x = _tokens(dev, B, H, dk, dv, q, k, v, alpha)
    op = _on(dev, out, "out", _OUT, (B, H, dv))
    epi = None
    if gate is not None:
        epi = ctypes.byref(kda_epilogue(_on(dev, gate, "gate", _BF16_TYPES, (B, H, dv)),
                                        None if weight is None else _on(dev, weight, "weight", _F32, (dv,)),
                                        float(eps)))
    elif weight is not None:
        raise ValueError("weight needs a gate")
    err = None if dev_err is None else _on(dev, dev_err, "dev_err", _I32, dev_err.shape)
    _call(dev, load_library().kda_lin_decode_step, "kda_lin_decode_step", cache.data_ptr(), ns, stride, slots,
          B, H, dk, dv, x, op, epi, err, _options(tile_w, out), _stream_of(dev, stream))


@functools.lru_cache(maxsize=1024)
def kda_lin_prefill_workspace(B: int, n_tok: int, H: int, dk: int, dv: int) -> int:
    """Workspace bytes kda_lin_prefill needs for these sizes (0: none)."""
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
    kda_lin_prefill_workspace() bytes; None allocates one for the call."""
    dev, ns, stride, H, dv, dk = _cache(cache)
    B = slot_ids.shape[0]
    slots = _on(dev, slot_ids, "slot_ids", _I32, (B,))
    cu = _on(dev, cu_seqlens, "cu_seqlens", _I32, (B + 1,))
    n_tok = v.shape[0]
    x = _tokens(dev, n_tok, H, dk, dv, q, k, v, alpha)
    op = _on(dev, out, "out", _OUT, (n_tok, H, dv))
    pos = ck = None
    if ckpt_pos is not None:
        pos = _on(dev, ckpt_pos, "ckpt_pos", _I32, (B,))
        if ckpt is None:
            raise ValueError("ckpt_pos needs a ckpt buffer")
    if ckpt is not None:
        ck = _on(dev, ckpt, "ckpt", _F32, (B, H, dv, dk))
    err = None if dev_err is None else _on(dev, dev_err, "dev_err", _I32, dev_err.shape)
    handle = _stream_of(dev, stream)
    if workspace is None:
        need = kda_lin_prefill_workspace(B, n_tok, H, dk, dv)
        if need and stream is not None:
            # allocated on the stream that uses it, so that its reuse is ordered behind the call
            with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=dev)):
                workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
        ws, nbytes = (workspace.data_ptr(), need) if need else (None, 0)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on GPU {dev}")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(dev, load_library().kda_lin_prefill, "kda_lin_prefill", cache.data_ptr(), ns, stride, slots, cu, B,
          n_tok, H, dk, dv, x, op, pos, ck, ws, nbytes, err, _options(0, out), handle)
