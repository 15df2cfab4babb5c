"""Python binding of the operators around a paged key/value cache: the norm and
rotation of queries and keys, appending to the cache, and differential attention
over it for new tokens and for trees of drafted tokens.

Only marshalling happens here, and little of it: a decode step makes these calls for
every layer, so descriptors are packed with one struct.pack and passed as bytes.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.DIFFATTN_BF16, torch.float32: _lib.DIFFATTN_F32}
_NO_STRIDE = (0, 0, 0)
# native alignment, as the C structs
_ROTARY = struct.Struct("@5q4ifiq2q2q24q")
_PAGES = struct.Struct("@4q9q")
_PAGED = struct.Struct("@5q2i9q2q")
assert _ROTARY.size == ctypes.sizeof(_lib.DiffattnRotaryDesc)
assert _PAGES.size == ctypes.sizeof(_lib.DiffattnPages)
assert _PAGED.size == ctypes.sizeof(_lib.DiffattnPagedDesc)


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


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t, name: str, dim: int, dtype, dev) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
    if t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")


def _inner(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _on_device:
    """torch.cuda.device(dev), skipped when it is the current one."""

    __slots__ = ("dev", "guard")

    def __init__(self, dev):
        self.dev = dev
        self.guard = None

    def __enter__(self):
        if torch.cuda.current_device() != self.dev.index:
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _weight(w, name: str, heads: int, D: int, dev):
    """(float32 dense weight or None, its head stride)."""
    if w is None:
        return None, 0
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if w.device != dev or tuple(w.shape) not in ((D,), (heads, D)):
        raise ValueError(f"{name} must be [D] = {(D,)} or [heads, D] = {(heads, D)} on the inputs' device")
    if not w.is_floating_point():
        raise ValueError(f"{name} must be a floating tensor")
    w32 = w.detach()
    if w32.dtype != torch.float32 or not w32.is_contiguous():
        w32 = w32.float().contiguous()
    return w32, D if w.dim() == 2 else 0


def _tables(cos, sin, D: int, dev):
    """(cos, sin, rotary_dim, rows); both None: no rotation."""
    if cos is None and sin is None:
        return None, None, 0, 0
    for n, t in (("cos", cos), ("sin", sin)):
        _need(t, n, 2, torch.float32, dev)
    if cos.shape != sin.shape or cos.shape[0] < 1 or cos.shape[1] < 1 or 2 * cos.shape[1] > D:
        raise ValueError("cos and sin must be [rows, rotary_dim / 2] with rotary_dim <= D, "
                         f"got {tuple(cos.shape)} and {tuple(sin.shape)}")
    if cos.requires_grad or sin.requires_grad:
        raise ValueError("cos and sin take no gradient")
    return cos.contiguous(), sin.contiguous(), 2 * cos.shape[1], cos.shape[0]


def _positions(positions, B: int, T: int, dev):
    """(positions or None, is int64, strides along B and T)."""
    if positions is None:
        return None, 0, (0, 0)
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if positions.device != dev or positions.dtype not in (torch.int32, torch.int64) or \
            tuple(positions.shape) not in ((B, T), (T,)):
        raise ValueError(f"positions must be an int32 or int64 tensor [T] or [B, T] = {(B, T)} on the inputs' device")
    s = positions.stride()
    return positions, int(positions.dtype == torch.int64), s if positions.dim() == 2 else (0, s[0])


_QK_NORMS = {None: _lib.DIFFATTN_NORM_NONE, "none": _lib.DIFFATTN_NORM_NONE, "rms": _lib.DIFFATTN_NORM_RMS}


def _qk_norm(norm, eps) -> int:
    if norm not in _QK_NORMS:
        raise ValueError(f"norm must be None, 'none' or 'rms', got {norm!r}")
    if _QK_NORMS[norm] and not 0 < eps < float("inf"):
        raise ValueError("norm_eps must be positive and finite")
    return _QK_NORMS[norm]


class _RotaryCall:
    """The checked arguments of one qk_norm_rotary call, for its forward and backward."""

    def __init__(self, xs, cos, sin, positions, norm, norm_eps, q_weight, k_weight, interleaved):
        given = [t for t in xs if t is not None]
        if not given:
            raise ValueError("at least one of q1, k1, q2, k2 must be given")
        first = given[0]
        for n, t in zip(("q1", "k1", "q2", "k2"), xs):
            if t is not None:
                _need(t, n, 4, first.dtype, first.device)
        if first.dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {first.dtype}; expected bfloat16 or float32")
        B, _, T, D = first.shape
        if B < 1 or T < 1 or not 1 <= D <= 128:
            raise ValueError(f"rows must be [B, heads, T, D] with B, T >= 1 and D <= 128, got {tuple(first.shape)}")
        heads = [None, None]
        for i, t in enumerate(xs):
            if t is None:
                continue
            if t.shape[0] != B or t.shape[2] != T or t.shape[3] != D or t.shape[1] < 1 or \
                    heads[i & 1] not in (None, t.shape[1]):
                raise ValueError("q1, q2 must share one shape [B, H, T, D], and k1, k2 [B, H_kv, T, D]")
            heads[i & 1] = t.shape[1]
        dev = first.device
        self.shape, self.dev, self.dtype = (B, T, D), dev, first.dtype
        self.heads = (heads[0] or 0, heads[1] or 0)
        self.cos, self.sin, self.R, self.rows = _tables(cos, sin, D, dev)
        self.pos, self.pos64, self.pos_stride = _positions(positions, B, T, dev)
        self.norm, self.eps = _qk_norm(norm, norm_eps), float(norm_eps)
        if not self.norm and (q_weight is not None or k_weight is not None):
            raise ValueError("q_weight and k_weight need norm='rms'")
        self.qw, self.qws = _weight(q_weight, "q_weight", self.heads[0], D, dev)
        self.kw, self.kws = _weight(k_weight, "k_weight", self.heads[1], D, dev)
        self.interleaved = int(bool(interleaved))

    def desc(self, xs, grads=(None,) * 4) -> bytes:
        B, T, D = self.shape
        s = []
        for t in (*xs, *grads):
            s += _NO_STRIDE if t is None else t.stride()[:3]
        return _ROTARY.pack(B, T, D, *self.heads, _DTYPES[self.dtype], self.R, self.interleaved, self.norm, self.eps,
                            self.pos64, self.rows, *self.pos_stride, self.qws, self.kws, *s)

    def forward(self, xs):
        outs = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=self.dev) for t in xs]
        lib = _lib.load()
        with _on_device(self.dev) as stream:
            rc = lib.diffattn_rotary(self.desc(xs), *map(_ptr, xs), _ptr(self.qw), _ptr(self.kw), _ptr(self.cos),
                                     _ptr(self.sin), _ptr(self.pos), *map(_ptr, outs), stream)
        _lib.check(rc, "diffattn_rotary")
        return outs

    def backward(self, xs, grads, want_qw: bool, want_kw: bool):
        dxs = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=self.dev) for t in xs]
        dqw = torch.empty_like(self.qw) if want_qw else None
        dkw = torch.empty_like(self.kw) if want_kw else None
        lib = _lib.load()
        desc = self.desc(xs, grads)
        with _on_device(self.dev) as stream:
            need = lib.diffattn_rotary_bwd_workspace_bytes(desc)
            ws = torch.empty(need, dtype=torch.uint8, device=self.dev)
            rc = lib.diffattn_rotary_bwd(desc, *map(_ptr, xs), _ptr(self.qw), _ptr(self.kw), _ptr(self.cos),
                                         _ptr(self.sin), _ptr(self.pos), *map(_ptr, grads), *map(_ptr, dxs),
                                         _ptr(dqw), _ptr(dkw), ws.data_ptr(), need, stream)
        _lib.check(rc, "diffattn_rotary_bwd")
        return dxs, dqw, dkw


class _RotaryFn(torch.autograd.Function):
    """Autograd node: forward through diffattn_rotary, backward through
    diffattn_rotary_bwd."""

    @staticmethod
    def forward(ctx, call, q1, k1, q2, k2, q_weight, k_weight):
        xs = [None if t is None else _inner(t.detach()) for t in (q1, k1, q2, k2)]
        outs = call.forward(xs)
        ctx.call = call
        # the norm's gradient needs the rows; the rotation's alone only their shapes
        ctx.save_for_backward(*xs, q_weight, k_weight, call.qw, call.kw, call.cos, call.sin, call.pos)
        return tuple(outs)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        call = ctx.call
        *xs, q_weight, k_weight = ctx.saved_tensors[:6]
        # saved_tensors checks that nothing saved was changed in place; the call holds the rest
        gs = []
        for x, g in zip(xs, grads):
            if x is None:
                gs.append(None)
            elif g is None:
                gs.append(torch.zeros(x.shape, dtype=x.dtype, device=x.device))
            else:
                gs.append(_inner(g.to(x.dtype)))
        want_qw = q_weight is not None and ctx.needs_input_grad[5]
        want_kw = k_weight is not None and ctx.needs_input_grad[6]
        dxs, dqw, dkw = call.backward(xs, gs, want_qw, want_kw)
        return (None, *dxs, dqw.to(q_weight.dtype) if want_qw else None, dkw.to(k_weight.dtype) if want_kw else None)


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
    None = 1.  Arithmetic in float32, one rounding at the end.

    Returns (q1, k1, q2, k2), contiguous, None where None was given.  Differentiable
    in the rows and the weights.  (Captured into a CUDA graph, take gradients with
    torch.autograd.grad, or with leaves that no eager graph still holds: torch's
    gradient accumulation otherwise joins the capture to the other graph's stream.)
    """
    shared = k2 is not None and k2 is k1
    xs = (q1, k1, q2, None if shared else k2)
    call = _RotaryCall(xs, cos, sin, positions, norm, norm_eps, q_weight, k_weight, interleaved)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (*xs, q_weight, k_weight)):
        outs = _RotaryFn.apply(call, *xs, q_weight, k_weight)
    else:
        outs = call.forward([None if t is None else _inner(t) for t in xs])
    return outs[0], outs[1], outs[2], outs[1] if shared else outs[3]


class _Cache:
    """The checked tensors of a paged cache."""

    __slots__ = ("k1", "k2", "v", "table", "shared", "desc", "Hk", "D", "Dv", "dev", "dtype", "B")

    def __init__(self, k1, k2, v, table, B: int):
        _need(k1, "k1_cache", 4, None, None)
        dev, dt = k1.device, k1.dtype
        if dt not in _DTYPES:
            raise ValueError(f"unsupported dtype {dt}; expected bfloat16 or float32")
        self.shared = k2 is None or k2 is k1
        if not self.shared:
            _need(k2, "k2_cache", 4, dt, dev)
            if k2.shape != k1.shape:
                raise ValueError(f"k1_cache and k2_cache must have one shape, got {tuple(k1.shape)}, {tuple(k2.shape)}")
        _need(v, "v_cache", 4, dt, dev)
        _need(table, "block_table", 2, torch.int32, dev)
        pages, self.Hk, page, self.D = k1.shape
        self.Dv = v.shape[3]
        if tuple(v.shape[:3]) != (pages, self.Hk, page) or min(k1.shape) < 1 or self.D > 128 or \
                not 1 <= self.Dv <= 256:
            raise ValueError("expected k1_cache, k2_cache [pages, H_kv, page_size, D], v_cache [pages, H_kv, "
                             f"page_size, Dv], D <= 128, Dv <= 256, got {tuple(k1.shape)}, {tuple(v.shape)}")
        if table.shape[0] != B or table.shape[1] < 1:
            raise ValueError(f"block_table must be [B, max_pages] with B = {B}, got {tuple(table.shape)}")
        for n, t in (("k1_cache", k1), ("k2_cache", k2), ("v_cache", v), ("block_table", table)):
            # a copy would not be the cache
            if t is not None and t.stride(-1) != 1 and t.shape[-1] != 1:
                raise ValueError(f"{n} must have a contiguous innermost dimension")
        self.k1, self.k2, self.v, self.table = k1, k1 if self.shared else k2, v, table
        self.dev, self.dtype, self.B = dev, dt, B
        self.desc = _PAGES.pack(pages, page, table.shape[1], table.stride(0), *k1.stride()[:3],
                                *self.k2.stride()[:3], *v.stride()[:3])

    def lengths(self, t, name: str):
        if t is None:
            return None
        _need(t, name, 1, torch.int32, self.dev)
        if t.shape[0] != self.B:
            raise ValueError(f"{name} must be [B] = {(self.B,)}, got {tuple(t.shape)}")
        return t.contiguous()


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
    written (None: all T).  positions: for the rotation, None = the index.
    A token whose index, page or position is out of range is not written and is
    reported by get_device_error.  Forward only."""
    _need(k1, "k1", 4, None, None)
    B, Hk, T, D = k1.shape
    c = _Cache(k1_cache, k2_cache, v_cache, block_table, B)
    if c.shared != (k2 is None or k2 is k1):
        raise ValueError("k2 and k2_cache must both be shared with k1 and k1_cache, or neither")
    ks = (k1,) if c.shared else (k1, k2)
    for n, t in zip(("k1", "k2"), ks):
        _need(t, n, 4, c.dtype, c.dev)
        if tuple(t.shape) != (B, c.Hk, T, c.D):
            raise ValueError(f"{n} must be [B, H_kv, T, D] with the cache's H_kv and D, got {tuple(t.shape)}")
    _need(value, "value", 4, c.dtype, c.dev)
    if tuple(value.shape) != (B, c.Hk, T, c.Dv) or T < 1:
        raise ValueError(f"value must be [B, H_kv, T, Dv] = {(B, c.Hk, T, c.Dv)}, got {tuple(value.shape)}")
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (*ks, value, k1_cache, k2_cache, v_cache, k_weight)):
        raise ValueError("paged_cache_append is forward only: call it under torch.no_grad() or detach its inputs")
    ks = [_inner(t) for t in ks]
    value = _inner(value)
    lengths = c.lengths(lengths, "lengths")
    if lengths is None:
        raise TypeError("lengths must be a torch.Tensor")
    new_lengths = c.lengths(new_lengths, "new_lengths")
    cos, sin, R, rows = _tables(cos, sin, D, c.dev)
    pos, pos64, pos_stride = _positions(positions, B, T, c.dev)
    code = _qk_norm(norm, norm_eps)
    if not code and k_weight is not None:
        raise ValueError("k_weight needs norm='rms'")
    kw, kws = _weight(k_weight, "k_weight", Hk, D, c.dev)
    k2s = ks[-1].stride()[:3]
    desc = _ROTARY.pack(B, T, D, 0, Hk, _DTYPES[c.dtype], R, int(bool(interleaved)), code, float(norm_eps), pos64,
                        rows, *pos_stride, 0, kws, *_NO_STRIDE, *ks[0].stride()[:3], *_NO_STRIDE, *k2s,
                        *(_NO_STRIDE * 4))
    lib = _lib.load()
    with _on_device(c.dev) as stream:
        rc = lib.diffattn_paged_append(desc, c.Dv, struct.pack("@3q", *value.stride()[:3]), c.desc, ks[0].data_ptr(),
                                       None if c.shared else ks[1].data_ptr(), value.data_ptr(), _ptr(kw), _ptr(cos),
                                       _ptr(sin), _ptr(pos), lengths.data_ptr(), _ptr(new_lengths),
                                       c.table.data_ptr(), c.k1.data_ptr(), None if c.shared else c.k2.data_ptr(),
                                       c.v.data_ptr(), stream)
    _lib.check(rc, "diffattn_paged_append")


def _paged_attention(q1, q2, cache, lengths, q_lengths, tree_mask, coefficient, out, norm, norm_eps, norm_weight,
                     norm_bias, out_scale):
    from . import _coefficient, _epilogue
    _need(q1, "q1", 4, None, None)
    B, H, Tq, D = q1.shape
    c = _Cache(*cache, B)
    for n, t in (("q1", q1), ("q2", q2)):
        _need(t, n, 4, c.dtype, c.dev)
        if tuple(t.shape) != (B, H, Tq, c.D) or H % c.Hk != 0 or H < 1 or B < 1:
            raise ValueError(f"{n} must be [B, H, Tq, D] with the cache's D and H_kv dividing H, got {tuple(t.shape)}")
    if not 1 <= Tq <= 1024:
        raise ValueError(f"1 to 1024 new tokens a call, got {Tq}")
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad
                                       for t in (q1, q2, *cache[:3], coefficient)):
        raise ValueError("attention over a paged cache is forward only: call it under torch.no_grad() or detach its "
                         "inputs")
    q1, q2 = _inner(q1), _inner(q2)
    lengths = c.lengths(lengths, "lengths")
    if lengths is None:
        raise TypeError("lengths must be a torch.Tensor")
    q_lengths = c.lengths(q_lengths, "q_lengths")
    mask_stride = (0, 0)
    if tree_mask is not None:
        if Tq > 64:
            raise ValueError(f"a tree holds up to 64 drafted tokens, got {Tq}")
        if not isinstance(tree_mask, torch.Tensor):
            raise TypeError("tree_mask must be a torch.Tensor")
        if tree_mask.device != c.dev or tree_mask.dtype != torch.bool or \
                tuple(tree_mask.shape) not in ((B, Tq, Tq), (Tq, Tq)):
            raise ValueError(f"tree_mask must be a bool tensor [B, Tq, Tq] or [Tq, Tq] = {(Tq, Tq)} on the cache's "
                             "device")
        tree_mask = _inner(tree_mask)
        s = tree_mask.stride()
        mask_stride = (s[0], s[1]) if tree_mask.dim() == 3 else (0, s[0])
    if out is None:
        # rows past a sequence's queries are left alone: they are zeros in a fresh output
        new = torch.empty if q_lengths is None else torch.zeros
        out = new((B, H, Tq, c.Dv), dtype=c.dtype, device=c.dev)
    else:
        _need(out, "out", 4, c.dtype, c.dev)
        if tuple(out.shape) != (B, H, Tq, c.Dv) or (out.stride(-1) != 1 and c.Dv != 1):
            raise ValueError("out must be [B, H, Tq, Dv] with a contiguous innermost dimension")
    lam, lam_dev = _coefficient(coefficient, c.dev)
    epi = _epilogue(norm, norm_eps, norm_weight, norm_bias, out_scale, H, c.Dv, c.dev)
    desc = _PAGED.pack(B, H, Tq, D, c.Dv, _DTYPES[c.dtype], H // c.Hk, *q1.stride()[:3], *q2.stride()[:3],
                       *out.stride()[:3], *mask_stride)
    lib = _lib.load()
    with _on_device(c.dev) as stream:
        need = lib.diffattn_paged_workspace_bytes(desc, c.desc)
        # from torch's allocator for every call: calls on other streams, and graphs
        # captured one after another, never share it
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=c.dev)
        rc = lib.diffattn_paged_decode(desc, c.desc, q1.data_ptr(), c.k1.data_ptr(), q2.data_ptr(), c.k2.data_ptr(),
                                       c.v.data_ptr(), c.table.data_ptr(), lengths.data_ptr(), _ptr(q_lengths),
                                       _ptr(tree_mask), lam, _ptr(lam_dev),
                                       ctypes.byref(epi[0]) if epi else None, out.data_ptr(), ws.data_ptr(),
                                       ws.numel(), stream)
    _lib.check(rc, "diffattn_paged_decode")
    return out


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
    rows of `out` past them are left as they were (zeros in a fresh output).
    coefficient and the epilogue (norm .. out_scale) as differential_attention.

    A length, or a page that a sequence needs, out of range gives that sequence rows
    of NaN and is reported by get_device_error.  Returns [B, H, Tq, Dv].  Forward only."""
    return _paged_attention(q1, q2, (k1_cache, k2_cache, v_cache, block_table), lengths, q_lengths, None, coefficient,
                            out, norm, norm_eps, norm_weight, norm_bias, out_scale)


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
    return _paged_attention(q1, q2, (k1_cache, k2_cache, v_cache, block_table), lengths, q_lengths, tree_mask,
                            coefficient, out, norm, norm_eps, norm_weight, norm_bias, out_scale)
