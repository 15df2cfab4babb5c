"""Python binding of the operators of a cross-attention block beside its rotation: the norm
of each head's output, with its gradients.

The arguments are checked and marshalled in C++ (csrc/binding.cpp), as those of the
operators around a paged cache.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _paged


def differential_head_norm(x: torch.Tensor, norm: str = "rms", norm_eps: float = 1e-5,
                           norm_weight: Optional[torch.Tensor] = None, norm_bias: Optional[torch.Tensor] = None,
                           out_scale: float = 1.0) -> torch.Tensor:
    """The step after the operation, as an operator of its own: the norm of each head's
    output over its channels, what differential_attention's epilogue does, with gradients.

    x: [B, H, T, Dv], bfloat16 or float32, Dv <= 256 (other strides than the innermost pass
    through: [B, T, H, Dv] seen as [B, H, T, Dv] needs no copy).  norm: "rms", or "group"
    (the mean of the row comes off first: a layer norm of every head).  norm_weight,
    norm_bias: [H, Dv] or [H * Dv], of any floating type, None = 1 and 0.  out_scale is
    applied last (1 - lambda_init).  float32 arithmetic, one rounding at the end.

    Returns [B, H, T, Dv], laid out as x where x is dense in some order of its dimensions.
    Differentiable in x, norm_weight and norm_bias, backward and once (what qk_norm_rotary
    says of captured backward passes and of forward mode holds here too)."""
    return (_paged._native or _paged._load()).head_norm(x, norm, norm_eps, norm_weight, norm_bias, out_scale)
