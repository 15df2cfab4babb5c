"""Plain float64 implementations of the paged-cache operators, and the error bounds
that the tests hold the kernels to.

Bounds.  A rounding is off by at most half a step, h = finfo(dtype).eps / 2 relative
to the value (bf16 2^-8, float32 2^-24); u = 2^-24 is float32's.

Norm and rotation: the arithmetic is float32 with one rounding at the end.  Of a row x
with r = (mean x^2 + eps)^-1/2, r is off by at most (D / 2 + 4) u relative (a sum of D
squares in any order, a division, a root, an inverse), each n by two more roundings and
each y = n_a cos - n_b sin by three: |y - y*| <= h |y*| + (D / 2 + 10) u (|n_a| + |n_b|).

Attention: with A_b the weights and S = A_1 |V| + |lambda| A_2 |V| (elementwise),
  bf16: each weight enters the product with V as two bf16 parts, the second the rounded
        rest of the first: h^2 S in all; the output is rounded once, h (|o| + the rest);
  both: a score is off by D u sum_i |q_i k_i| / sqrt(D) (a sum of D products) and two
        roundings of scale and maximum, its exponential by 4 u more, and sums over n
        keys by n u relative: each weight by
        e = u (n + 2 D z + 2 z + 16), z the row's largest sum_i |q_i k_i| / sqrt(D).
        Both the weights and their sum have that error: 2 e S, and 4 u S for the rest.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_rotate(x, w, cos, sin, pos, interleaved, norm, eps):
    """x [B, H, T, D] float64, w [D], [H, D] or None, cos/sin [P, R/2] or None, pos [B, T].
    Returns (y, bound of y without its rounding)."""
    D = x.shape[-1]
    n = x
    if norm:
        n = n / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            n = n * (w if w.dim() == 1 else w[None, :, None, :])
    y, size = n.clone(), n.abs()
    if cos is not None:
        R = 2 * cos.shape[1]
        i = torch.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = cos[pos][:, None], sin[pos][:, None]
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        size[..., a] = size[..., b] = n[..., a].abs() + n[..., b].abs()
    return y, (D / 2 + 10) * U * size


def norm_rotate_backward(x, w, cos, sin, pos, interleaved, norm, eps, dy):
    """(dx, dw per head [H, D] or None, sums of |terms| of dw)."""
    u = dy.clone()
    if cos is not None:
        R = 2 * cos.shape[1]
        i = torch.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = cos[pos][:, None], sin[pos][:, None]
        u[..., a] = dy[..., a] * c + dy[..., b] * s
        u[..., b] = dy[..., b] * c - dy[..., a] * s
    if not norm:
        return u, None, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    terms = u * x * r
    g = u if w is None else u * (w if w.dim() == 1 else w[None, :, None, :])
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx, terms.sum((0, 2)), terms.abs().sum((0, 2))


def visible(before, n_new, tree):
    """[n_new, before + n_new] bool; tree [n_new, n_new] bool or None (causal)."""
    new = torch.ones(n_new, n_new, dtype=torch.bool).tril() if tree is None else tree
    return torch.cat([torch.ones(n_new, before, dtype=torch.bool), new], 1)


def attention_rows(q1, k1, q2, k2, v, seen, lam, dtype):
    """One sequence and head in float64: q [t, D], k [n, D], v [n, Dv], seen [t, n].
    Returns (o, bound).  A row that sees nothing is 0; hidden keys and values take no part."""
    t, n, D = q1.shape[0], k1.shape[0], q1.shape[1]
    o, size, e = 0, 0, 0
    for q, k, f in ((q1, k1, 1.0), (q2, k2, -lam)):
        s = (q @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        a = torch.exp(s - torch.where(torch.isneginf(top), torch.zeros_like(top), top)).masked_fill(~seen, 0.0)
        a = a / a.sum(-1, keepdim=True).clamp(min=1e-300)
        # products with hidden values left out, whatever they hold
        prod = torch.where(seen[:, :, None], a[:, :, None] * v[None], torch.zeros((), dtype=v.dtype))
        o = o + f * prod.sum(1)
        size = size + abs(f) * prod.abs().sum(1)
        z = (q.abs() @ k.abs().T / math.sqrt(D)).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
        e = torch.maximum(torch.as_tensor(e, dtype=v.dtype), U * (n + 2 * D * z + 2 * z + 16))
    h = half_step(dtype)
    parts = h * h if dtype == torch.bfloat16 else 0.0
    return o, (1 + h) * (2 * e + 4 * U + parts) * size + h * o.abs()


def epilogue(o, bound, norm, eps, weight, bias, scale, dtype):
    """The per-head epilogue of o [t, Dv] and its bound: with rho = (mean o^2 + eps)^1/2
    (of o - mean for "group"), an error d of o changes y by at most (|d| + mean|d|) |w| / rho
    and rho by rms(d) relative to itself; one rounding at the end, 8 float32 ones before."""
    base = bound - half_step(dtype) * o.abs()           # the rounding is the epilogue's
    x, d = o, base
    if norm == "group":
        x = o - o.mean(-1, keepdim=True)
        d = base + base.mean(-1, keepdim=True)
    if norm in ("rms", "group"):
        rho = torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        rel = torch.sqrt((d * d).mean(-1, keepdim=True)) / rho + (x.shape[-1] / 2 + 8) * U
        x, d = x / rho, d / rho + (x / rho).abs() * rel
    y = x if weight is None else x * weight
    d = d if weight is None else d * weight.abs()
    if bias is not None:
        y = y + bias
    y = scale * y
    return y, abs(scale) * d + 8 * U * y.abs() + half_step(dtype) * y.abs()
