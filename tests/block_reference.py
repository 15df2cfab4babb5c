"""The operators of a cross-attention block from their formulas, in float64 on the CPU, with
the sizes that their tests' error bounds go by."""
import torch


def head_norm(x, group, eps, w, b, scale):
    """y [B, H, T, C], and h, r, mean |x| of its rows; w, b [H, C] or None."""
    size = x.abs().mean(-1, keepdim=True)
    if group:
        x = x - x.mean(-1, keepdim=True)
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    h = x * r
    y = h if w is None else h * w[:, None]
    if b is not None:
        y = y + b[:, None]
    return scale * y, h, r, size


def head_norm_backward(x, group, eps, w, scale, dy):
    """dx, dw [H, C], db [H, C]."""
    _, h, r, _ = head_norm(x, group, eps, None, None, 1.0)
    g = scale * (dy if w is None else dy * w[:, None])
    dx = g - h * (g * h).mean(-1, keepdim=True)
    if group:
        dx = dx - g.mean(-1, keepdim=True)
    return r * dx, scale * (dy * h).sum((0, 2)), scale * dy.sum((0, 2))
