"""Python binding of the operators of a cross-attention block beside its rotation: attention
over an encoder's states and the norm of each head's output, with their gradients.

The arguments are checked and marshalled in C++ (csrc/binding.cpp), as those of the
operators around a paged cache.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _paged


def differential_cross_attention(q1: torch.Tensor, k1: torch.Tensor, q2: torch.Tensor, k2: Optional[torch.Tensor],
                                 value: torch.Tensor, coefficient, kv_lengths: Optional[torch.Tensor] = None,
                                 out: Optional[torch.Tensor] = None, norm: Optional[str] = None, norm_eps: float = 1e-5,
                                 norm_weight: Optional[torch.Tensor] = None, norm_bias: Optional[torch.Tensor] = None,
                                 out_scale: float = 1.0) -> torch.Tensor:
    """Differential attention over an encoder's states of another length, without a causal
    mask: in training, over a whole target sequence, and in serving, a token at a time.

    q1, q2: [B, H, Tq, D]; k1, k2: [B, H_kv, Tk, D], value: [B, H_kv, Tk, Dv], the encoder's
    states as the layer projected them, H_kv dividing H, D <= 128, Dv <= 256; bfloat16 or
    float32; other strides than the innermost pass through.  k2 None or k1 again (the same
    object): one key tensor for both branches.  kv_lengths: [B] int32 on the device, sequence b
    has only its first kv_lengths[b] states (None: all Tk), and what lies behind them has no
    influence, NaN included; one with none gives zeros (before the epilogue).  coefficient, out
    and the epilogue (norm .. out_scale) as differential_attention, norm_weight and norm_bias
    with a norm alone; out may not overlap the inputs.

    The tensor cores take bfloat16 with Dv = 128 and D = 64 or 128, in training D = 128 with one
    key tensor.  Inputs whose rows have a stride of 0 or are not of whole 16-byte pieces are
    copied for them, beyond a few rows.  Other widths, an out of such rows, and a training step
    of more than 65535 sequences times heads run on the CUDA cores, about forty times slower.

    Returns [B, H, Tq, Dv].  In bfloat16 the weights keep 16 bits on every path, so that what
    branches that cancel leave is off by its own rounding alone.  Differentiable in q1, q2, k1,
    k2, value and a tensor coefficient, backward and once, without out and the epilogue
    (differential_head_norm has gradients); states that a sequence does not have get zeros.  What
    qk_norm_rotary says of captured backward passes and of forward mode holds here too.  A
    length outside 0 .. Tk gives that sequence rows (and gradients) of NaN and is reported by get_device_error."""
    return (_paged._native or _paged._load()).cross(q1, k1, q2, k2, value, coefficient, kv_lengths, out, norm, norm_eps,
                                                    norm_weight, norm_bias, out_scale)


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
