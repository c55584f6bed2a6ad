"""Python binding of include/kda_norm.h: the norms around a block, fused with its
gate, residual scale and residual add.

    r' = r + res_scale * sigmoid(gate) * N(z) * w_post ;  y = N(r') * w_pre
    N(x) = x / sqrt(mean(x^2) + eps)
"""

from __future__ import annotations

from typing import Optional

import torch

from .kda import KDA_OK, KdaError
from .native import native

KDA_NORM_RESID_BF16 = 1
KDA_NORM_Y_BF16 = 2
KDA_NORM_MAX_D = 16384


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
    rc = native().block_norm(resid, z, resid_out, y, w_post, gate, res_scale, w_pre, eps, stream)
    if rc != KDA_OK:
        raise KdaError(rc, "kda_block_norm")
