"""Python binding of include/kda_norm.h: the norms around a block, fused with its
gate, residual scale and residual add.

    r' = r + res_scale * sigmoid(gate) * N(z) * w_post ;  y = N(r') * w_pre
    N(x) = x / sqrt(mean(x^2) + eps)
"""

from __future__ import annotations

from typing import Optional

import torch

from .kda import _BF16_TYPES, load_library
from .linear import _F32, _OUT, _call, _on, _refuse, _stream_of

KDA_NORM_RESID_BF16 = 1
KDA_NORM_Y_BF16 = 2
KDA_NORM_MAX_D = 16384


def _rows(dev: int, t, name: str, dtypes, rows: int, D: int):
    """(address, stride between rows) of a [rows, D] tensor whose rows are contiguous."""
    if t is None:
        return None, 0
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev and t.shape == (rows, D)):
        _refuse(dev, t, name, dtypes, (rows, D))
    s = t.stride()
    if D > 1 and s[1] != 1:
        raise ValueError(f"{name}: each row must be contiguous, got strides {s}")
    return t.data_ptr(), (s[0] if rows > 1 else D)


def kda_block_norm(resid: torch.Tensor, z: Optional[torch.Tensor] = None,
                   resid_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, *,
                   w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                   res_scale: float = 1.0, w_pre: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   stream=None) -> None:
    """resid_out <- resid + res_scale * sigmoid(gate) * N(z) * w_post, y <- N(that) * w_pre.

    resid, resid_out float32 or bf16 [rows, D] (the same type; resid_out may be resid); z, gate bf16
    [rows, D]; y float32 or bf16 [rows, D]; w_post, w_pre float32 [D]. Rows may be strided. Without
    w_post z is not normalized, without gate it is not gated, without z resid itself is normalized,
    without y (and w_pre) only resid_out is written.
    """
    if not isinstance(resid, torch.Tensor) or not resid.is_cuda or resid.dim() != 2:
        raise ValueError("resid must be a GPU tensor [rows, D]")
    dev = resid.get_device()
    rows, D = resid.shape
    rp, rs = _rows(dev, resid, "resid", _OUT, rows, D)
    zp, zs = _rows(dev, z, "z", _BF16_TYPES, rows, D)
    op, os_ = _rows(dev, resid_out, "resid_out", (resid.dtype,), rows, D)
    yp, ys = _rows(dev, y, "y", _OUT, rows, D)
    gp, gs = _rows(dev, gate, "gate", _BF16_TYPES, rows, D)
    wpost = None if w_post is None else _on(dev, w_post, "w_post", _F32, (D,))
    wpre = None if w_pre is None else _on(dev, w_pre, "w_pre", _F32, (D,))
    flags = (KDA_NORM_RESID_BF16 if resid.dtype is not torch.float32 else 0) | \
        (KDA_NORM_Y_BF16 if y is not None and y.dtype is not torch.float32 else 0)
    _call(dev, load_library().kda_block_norm, "kda_block_norm", rp, rs, zp, zs, op, os_, yp, ys, wpost, gp, gs,
          float(res_scale), wpre, float(eps), rows, D, flags, _stream_of(dev, stream))
