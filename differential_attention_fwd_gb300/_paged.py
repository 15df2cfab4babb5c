"""Python binding of the operators around a paged key/value cache: the norm and
rotation of queries and keys, appending to the cache, and differential attention
over it for new tokens and for trees of drafted tokens.

The arguments are checked and marshalled in C++ (csrc/binding.cpp): a decode step makes
these calls for every layer, and its kernels take a few microseconds.
"""
from __future__ import annotations

import importlib
import os
from typing import Optional

import torch

from . import _lib, build

_native = None


def _load():
    """The compiled binding (once).  Raises if it has not been built."""
    global _native
    if _native is None:
        _lib.load()
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")):
            raise RuntimeError("_binding.so is missing: build the CUDA library first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        made_for = build.binding_torch()
        if made_for not in (None, build.torch_version()):
            raise RuntimeError(f"_binding.so was built for torch {made_for}, and torch {build.torch_version()} is installed: "
                               "build it again (python -c 'import __graft_entry__ as g; g.build()')")
        _native = importlib.import_module("._binding", __package__)
        _native.set_error(_lib.DiffattnError)
    return _native


def rotary_tables(positions: int, rotary_dim: int, base: float = 10000.0, device=None):
    """(cos, sin) tables of the position rotation, float32 [positions,
    rotary_dim / 2]: entry (p, i) is the cosine (sine) of p * base^(-2 i /
    rotary_dim).  The angles are formed in float64, since a float32 angle is
    already off by 2^-8 at position 100,000.  Made once, at set-up."""
    if positions < 1 or rotary_dim < 2 or rotary_dim % 2 != 0:
        raise ValueError("positions must be at least 1 and rotary_dim even and at least 2")
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float(), a.sin().float()


def qk_norm_rotary(q1: Optional[torch.Tensor], k1: Optional[torch.Tensor], q2: Optional[torch.Tensor],
                   k2: Optional[torch.Tensor], cos: Optional[torch.Tensor], sin: Optional[torch.Tensor],
                   positions: Optional[torch.Tensor] = None, norm: Optional[str] = "rms", norm_eps: float = 1e-6,
                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                   interleaved: bool = False):
    """The step before the operation: the RMS norm of each query and key head and
    the rotation of its pairs by the token's position, in one launch.

    q1, q2: [B, H, T, D]; k1, k2: [B, H_kv, T, D]; bfloat16 or float32, D <= 128,
    innermost dimension contiguous (other strides pass through, so a projection's
    [B, T, heads, D] seen as [B, heads, T, D] needs no copy).  Any of them may be
    None (a decode step rotates its keys in paged_cache_append).  Passing the same
    tensor as k1 and k2 shares it: it is rotated once and returned twice.

    cos, sin: [positions, R / 2] float32 tables (rotary_tables); the first R <= D
    elements of a row are rotated, in pairs (i, i + R/2), or (2i, 2i + 1) with
    interleaved=True; None for both: no rotation.  positions: int32 or int64, [T] or
    [B, T]; None: 0 .. T-1.  A position outside the tables gives a row of NaN and is
    reported by get_device_error.
    norm: "rms" or None; q_weight and k_weight: [D] (for every head) or [heads, D],
    None = 1; one whose rows are left out is not used and gets no gradient.
    Arithmetic in float32, one rounding at the end.

    Returns (q1, k1, q2, k2), contiguous, None where None was given.  Differentiable
    in the rows and the weights, backward and once; dual tensors of forward-mode
    differentiation are refused, here and in the calls below.  (A backward pass captured into a CUDA graph must not
    add to leaves that an eager graph on the default stream still holds: torch would join
    that stream to the capture, so this is an error.  torch.autograd.grad is free of it.)
    """
    return (_native or _load()).rotary(q1, k1, q2, k2, cos, sin, positions, norm, norm_eps, q_weight, k_weight,
                                       interleaved)


def paged_cache_append(k1: torch.Tensor, k2: Optional[torch.Tensor], value: torch.Tensor, k1_cache: torch.Tensor,
                       k2_cache: Optional[torch.Tensor], v_cache: torch.Tensor, block_table: torch.Tensor,
                       lengths: torch.Tensor, new_lengths: Optional[torch.Tensor] = None,
                       cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                       positions: Optional[torch.Tensor] = None, norm: Optional[str] = None, norm_eps: float = 1e-6,
                       k_weight: Optional[torch.Tensor] = None, interleaved: bool = False) -> None:
    """Write new keys and values into a paged cache, in place, the keys normed and
    rotated on the way (arguments of qk_norm_rotary; by default neither).  One launch.

    k1, k2: [B, H_kv, T, D], value: [B, H_kv, T, Dv]: the new tokens' rows.
    k1_cache, k2_cache: [pages, H_kv, page_size, D], v_cache: [pages, H_kv, page_size,
    Dv]; block_table: [B, max_pages] int32, the page of each page_size tokens of a
    sequence.  k2 and k2_cache None (or k1 and k1_cache again): the branches share
    their keys.  lengths: [B] int32, tokens cached before the call; token t goes to
    index lengths[b] + t.  new_lengths: [B] int32, the first new_lengths[b] tokens are
    written (None: all T).  positions: for the rotation, None = the index.  No two
    tokens of a call may have one slot, and the new rows may not lie in the caches.
    A token whose index, page or position is out of range is not written and is
    reported by get_device_error.  Forward only."""
    (_native or _load()).append(k1, k2, value, k1_cache, k2_cache, v_cache, block_table, lengths, new_lengths, cos, sin,
                                positions, norm, norm_eps, k_weight, interleaved)


def differential_attention_paged(q1: torch.Tensor, k1_cache: torch.Tensor, q2: torch.Tensor,
                                 k2_cache: Optional[torch.Tensor], v_cache: torch.Tensor, block_table: torch.Tensor,
                                 lengths: torch.Tensor, coefficient, q_lengths: Optional[torch.Tensor] = None,
                                 out: Optional[torch.Tensor] = None, norm: Optional[str] = None,
                                 norm_eps: float = 1e-5, norm_weight: Optional[torch.Tensor] = None,
                                 norm_bias: Optional[torch.Tensor] = None, out_scale: float = 1.0) -> torch.Tensor:
    """Differential attention of new tokens over a paged cache.

    q1, q2: [B, H, Tq, D] (Tq 1 to 1024: a decode step, or a chunk of a prefill);
    the cache and block_table as in paged_cache_append, H_kv dividing H; k2_cache
    None or k1_cache again: one key tensor for both branches.  lengths: [B] int32,
    tokens cached before the new ones, as given to paged_cache_append, which has put
    the new tokens' keys and values behind them.  New token i of sequence b sees the
    lengths[b] tokens before and new tokens 0 .. i.  q_lengths: [B] int32, sequence b
    has only its first q_lengths[b] new tokens (0: an idle place of the batch): the
    rows of `out` past them are left as they were (zeros in a fresh output); it may not
    overlap the inputs.
    coefficient and the epilogue (norm .. out_scale) as differential_attention.

    A length, or a page that a sequence needs, out of range gives that sequence rows
    of NaN and is reported by get_device_error.  Returns [B, H, Tq, Dv].  Forward only."""
    return (_native or _load()).attention(q1, k1_cache, q2, k2_cache, v_cache, block_table, lengths, q_lengths, None,
                                          coefficient, out, norm, norm_eps, norm_weight, norm_bias, out_scale)


def differential_attention_tree(q1: torch.Tensor, k1_cache: torch.Tensor, q2: torch.Tensor,
                                k2_cache: Optional[torch.Tensor], v_cache: torch.Tensor, block_table: torch.Tensor,
                                lengths: torch.Tensor, tree_mask: torch.Tensor, coefficient,
                                q_lengths: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                norm: Optional[str] = None, norm_eps: float = 1e-5,
                                norm_weight: Optional[torch.Tensor] = None, norm_bias: Optional[torch.Tensor] = None,
                                out_scale: float = 1.0) -> torch.Tensor:
    """Differential attention for a tree of drafted tokens over a paged cache: as
    differential_attention_paged, with Tq up to 64 drafted tokens a sequence, whose
    keys and values are in the cache behind its lengths[b] tokens in any order, and
    tree_mask [B, Tq, Tq] (or [Tq, Tq] for all) bool: drafted token i sees drafted
    token j where it is true (itself and its ancestors).  Every drafted token sees the
    cached ones.  Nothing that a token does not see influences it; one that sees
    nothing at all gives zeros (before the epilogue)."""
    if tree_mask is None:
        raise TypeError("tree_mask must be a torch.Tensor")
    return (_native or _load()).attention(q1, k1_cache, q2, k2_cache, v_cache, block_table, lengths, q_lengths, tree_mask,
                                          coefficient, out, norm, norm_eps, norm_weight, norm_bias, out_scale)
