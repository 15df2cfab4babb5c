"""GPU tests of differential_head_norm against its formulas in float64.

The bounds count roundings.  u = 2^-24 is half a float32 step relative to its value; a
result rounded to bf16 is off by 2^-8 of itself, to float32 by u.  The sums over a row go
through at most 8 additions in a lane, 1 of a pair's halves and 5 between lanes (14);
with the products before them and the multiplication by 1 / C a mean is off by 16 u of
the mean of the magnitudes.  So mu is off by 16 u mean|x|, the sum of squares by 16 u of
itself (twice, with mu's error in it), r by half of that and by 4 u of rsqrt (2 units in
the last place) and 2 u of the additions and the root's argument; h = (x - mu) r by
24 u |h| + 16 u mean|x| r.  With the products by w and the scale K = 32 covers y.
"""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import block_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = 2.0 ** -24
K = 32 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _clean():
    da.get_device_error()
    yield
    assert da.get_device_error() == 0


def d64(t):
    return None if t is None else t.detach().cpu().double()


def check(name, got, want, tol):
    got = d64(got)
    assert got.shape == want.shape
    worst = ((got - want).abs() - tol).max()
    assert worst <= 0, f"{name}: {worst.item():.3g} beyond its bound"


def compare(x, norm, w, b, scale, dy, y, dx, dw, db):
    """All results against the formulas, each within its bound."""
    dt = x.dtype
    group = norm == "group"
    x, w_, b_, dy = d64(x), d64(w), d64(b), d64(dy)
    H, C = x.shape[1], x.shape[3]
    want, h, r, size = ref.head_norm(x, group, EPS, w_, b_, scale)
    one = torch.ones(H, C, dtype=torch.float64)
    aw = (one if w_ is None else w_.abs())[:, None]
    ab = 0 if b_ is None else b_.abs()[:, None]
    dh = K * (h.abs() + size * r)                       # h's error
    check("y", y, want, HALF[dt] * want.abs() + abs(scale) * (aw * dh + K * ab) + 1e-30)
    if dy is None:
        return
    wdx, wdw, wdb = ref.head_norm_backward(x, group, EPS, w_, scale, dy)
    g = abs(scale) * aw * dy.abs()
    mean = lambda t: t.mean(-1, keepdim=True)           # noqa: E731
    # g, its two means and h enter with their own errors, each by the others' sizes
    tol = r * (2 * K * (g + mean(g) + h.abs() * mean(g * h.abs())) + dh * mean(g * h.abs()) + h.abs() * mean(g * dh))
    tol = tol + 2 * K * wdx.abs() + 16 * U * (size * r) ** 2 * r * g            # r's own error through mu's
    if dx is not None:
        check("dx", dx, wdx, HALF[dt] * wdx.abs() + tol + 1e-30)
    n = x.shape[0] * x.shape[2] + 64                    # additions of a channel's sum, at most
    if dw is not None:
        check("dw", dw, wdw, abs(scale) * ((n * U) * (dy * h).abs().sum((0, 2)) + (dy.abs() * dh).sum((0, 2))) + 1e-30)
    if db is not None:
        check("db", db, wdb, abs(scale) * n * U * dy.abs().sum((0, 2)) + 1e-30)


def run(x, norm, w, b, scale, dy):
    leaves = [t for t in (x, w, b) if t is not None]
    for t in leaves:
        t.requires_grad_()
    y = da.differential_head_norm(x, norm=norm, norm_eps=EPS, norm_weight=w, norm_bias=b, out_scale=scale)
    grads = list(torch.autograd.grad(y, leaves, dy))
    dx = grads.pop(0)
    dw = grads.pop(0) if w is not None else None
    db = grads.pop(0) if b is not None else None
    return y, dx, dw, db


def inputs(seed, B, H, T, C, dtype, layout="bhtc", offset=0.0):
    g = torch.Generator().manual_seed(seed)

    def rows(shift=0.0):
        t = torch.randn(B, H, T, C, generator=g) + shift
        if layout == "bthc":
            return t.transpose(1, 2).contiguous().to(dtype).cuda().transpose(1, 2)
        if layout == "padded":                          # rows with a gap: not dense, and not on 16 bytes
            out = torch.full((B, H, T, C + 3), float("nan")).to(dtype).cuda()
            out[..., :C] = t.to(dtype).cuda()
            return out[..., :C]
        return t.to(dtype).cuda()
    return rows(offset), rows(), (1 + 0.3 * torch.randn(H, C, generator=g)).cuda(), (0.3 * torch.randn(H, C, generator=g)).cuda()


@pytest.mark.parametrize("norm", ["rms", "group"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [128, 64, 256, 32, 96, 8, 136, 1, 7, 100, 255])
def test_widths(norm, dtype, C):
    x, dy, w, b = inputs(C, 2, 3, 41, C, dtype)
    compare(x, norm, w, b, 0.2, dy, *run(x, norm, w, b, 0.2, dy))


@pytest.mark.parametrize("norm", ["rms", "group"])
@pytest.mark.parametrize("layout", ["bthc", "padded"])
@pytest.mark.parametrize("B,H,T", [(1, 1, 1), (1, 16, 1), (3, 5, 1), (1, 1, 1000), (2, 3, 517), (5, 2, 129)])
def test_sizes_and_layouts(norm, layout, B, H, T):
    for dtype in (torch.bfloat16, torch.float32):
        x, dy, w, b = inputs(T, B, H, T, 128, dtype, layout)
        y, dx, dw, db = run(x, norm, w, b, 1.0, dy)
        if layout == "bthc" and T > 1 and H > 1:
            assert y.stride() == x.stride() and dx.stride() == x.stride()
        if layout == "padded":
            assert y.is_contiguous()
        compare(x, norm, w, b, 1.0, dy, y, dx, dw, db)


def test_long_sums():
    """Chunks of many rows a block, and more blocks than one head has."""
    x, dy, w, b = inputs(5, 2, 2, 20000, 64, torch.float32)
    compare(x, "group", w, b, 0.7, dy, *run(x, "group", w, b, 0.7, dy))


def test_values_far_from_zero():
    x, dy, w, b = inputs(6, 1, 2, 50, 128, torch.float32, offset=300.0)
    compare(x, "group", w, b, 1.0, dy, *run(x, "group", w, b, 1.0, dy))


@pytest.mark.parametrize("which", ["x", "w", "b", "xb", "none"])
def test_some_parameters(which):
    """Gradients of what asks for them alone, and parameters left out."""
    x, dy, w, b = inputs(7, 2, 4, 33, 128, torch.bfloat16)
    leaves = [t.requires_grad_() for k, t in (("x", x), ("w", w), ("b", b)) if k in which]
    if which == "xb":
        w = None
    if which == "none":
        w = b = None
        leaves = [x.requires_grad_()]
    y = da.differential_head_norm(x, "rms", EPS, w, b, 0.5)
    got = dict(zip([k for k in "xwb" if k in which] or "x", torch.autograd.grad(y, leaves, dy)))
    compare(x, "rms", w, b, 0.5, dy, y, got.get("x"), got.get("w"), got.get("b"))


def test_parameters_of_other_types_and_shapes():
    x, dy, w, b = inputs(8, 2, 4, 33, 64, torch.bfloat16)
    w16 = w.bfloat16().reshape(-1).requires_grad_()
    b64 = b.double().requires_grad_()
    y = da.differential_head_norm(x, "group", EPS, w16, b64, 1.0)
    dw, db = torch.autograd.grad(y, [w16, b64], dy)
    assert dw.shape == w16.shape and dw.dtype == torch.bfloat16 and db.dtype == torch.float64
    w32, b32 = w16.detach().float().reshape(4, 64).requires_grad_(), b64.detach().float().requires_grad_()
    y2 = da.differential_head_norm(x, "group", EPS, w32, b32, 1.0)
    assert torch.equal(y, y2)
    ref_w, ref_b = torch.autograd.grad(y2, [w32, b32], dy)
    assert torch.equal(dw, ref_w.bfloat16().reshape(-1)) and torch.equal(db, ref_b.double())


def test_non_finite_rows_stay_their_own():
    x, dy, w, b = inputs(9, 1, 3, 40, 128, torch.float32)
    y0 = da.differential_head_norm(x, "group", EPS, w, b)
    x[0, 1, 7, 5] = float("nan")
    x[0, 2, 9] = float("inf")
    y = da.differential_head_norm(x, "group", EPS, w, b)
    assert y[0, 1, 7].isnan().all() and y[0, 2, 9].isnan().all()
    y[0, 1, 7], y[0, 2, 9] = y0[0, 1, 7], y0[0, 2, 9]
    assert torch.equal(y, y0)


def test_agrees_with_the_attention_epilogue():
    """differential_attention's fused epilogue and this operator on its bare float32 output."""
    g = torch.Generator().manual_seed(11)
    q1, k1, q2, k2 = (torch.randn(2, 3, 70, 32, generator=g).cuda() for _ in range(4))
    v = torch.randn(2, 3, 70, 64, generator=g).cuda()
    w, b = torch.randn(3, 64, generator=g).cuda(), torch.randn(3, 64, generator=g).cuda()
    for norm in ("rms", "group"):
        fused = da.differential_attention(q1, k1, q2, k2, v, 0.4, norm=norm, norm_eps=EPS, norm_weight=w, norm_bias=b, out_scale=0.2)
        o = da.differential_attention(q1, k1, q2, k2, v, 0.4)
        y = da.differential_head_norm(o, norm, EPS, w, b, 0.2)
        want, h, r, size = ref.head_norm(d64(o), norm == "group", EPS, d64(w), d64(b), 0.2)
        # either is within y's bound of the formulas (the fused one's sums have other orders: 64
        # additions of a lane's at most)
        tol = 0.2 * 4 * K * (d64(w).abs()[:, None] * (h.abs() + size * r) + d64(b).abs()[:, None]) + U * want.abs()
        check("fused", fused, want, tol)
        check("y", y, want, tol)


def test_training_step_through_attention_and_norm():
    """Attention, then the norm: the gradients reach Q, K, V and both parameters, and equal those
    of the two steps apart."""
    g = torch.Generator().manual_seed(12)
    q1, k1, q2, k2 = (torch.randn(1, 4, 130, 64, generator=g).bfloat16().cuda().requires_grad_() for _ in range(4))
    v = torch.randn(1, 4, 130, 128, generator=g).bfloat16().cuda().requires_grad_()
    w = torch.ones(4, 128, device="cuda", requires_grad=True)
    o = da.differential_attention(q1, k1, q2, k2, v, 0.8)
    y = da.differential_head_norm(o, "group", EPS, w, None, 0.2)
    dy = torch.randn(y.shape, generator=g).bfloat16().cuda()
    leaves = [q1, k1, q2, k2, v, w]
    grads = torch.autograd.grad(y, leaves, dy)
    o1 = o.detach().requires_grad_()
    do, dw = torch.autograd.grad(da.differential_head_norm(o1, "group", EPS, w, None, 0.2), [o1, w], dy)
    o2 = da.differential_attention(q1, k1, q2, k2, v, 0.8)
    apart = torch.autograd.grad(o2, leaves[:5], do)
    for a, e in zip(grads, (*apart, dw)):
        assert torch.equal(a, e)


def test_same_bits_each_time_and_on_another_stream():
    x, dy, w, b = inputs(13, 2, 16, 300, 128, torch.bfloat16)
    first = run(x, "group", w, b, 1.0, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = run(x, "group", w, b, 1.0, dy)
    s.synchronize()
    for p, q in zip(first, second):
        assert torch.equal(p, q)


def test_captured_and_replayed():
    x, dy, w, b = inputs(14, 2, 4, 100, 128, torch.bfloat16)
    x.requires_grad_()
    w.requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            torch.autograd.grad(da.differential_head_norm(x, "rms", EPS, w, None), [x, w], dy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = da.differential_head_norm(x, "rms", EPS, w, None)
        dx, dw = torch.autograd.grad(y, [x, w], dy)
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
        dy.copy_(torch.randn_like(dy))
    graph.replay()
    torch.cuda.synchronize()
    compare(x, "rms", w, None, 1.0, dy, y, dx, dw, None)


def test_captured_backward_beside_a_living_graph():
    """Gradients added in a capture to leaves that an eager graph on the default stream holds: torch
    would end the process, so this is refused.  Without that graph the same capture works."""
    x, dy, w, b = inputs(15, 1, 2, 10, 64, torch.float32)
    w.requires_grad_()
    eager = da.differential_head_norm(x, "rms", EPS, w)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="default stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            da.differential_head_norm(x, "rms", EPS, w).backward(dy)
    assert w.grad is None
    want = torch.autograd.grad(eager, w, dy)[0]
    del eager
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.differential_head_norm(x, "rms", EPS, w).backward(dy)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w.grad, want)


def test_refusals():
    x, dy, w, b = inputs(16, 1, 2, 10, 64, torch.float32)
    f = da.differential_head_norm
    for bad in (dict(norm=None), dict(norm="none"), dict(norm="layer"), dict(norm_eps=0.0), dict(norm_eps=float("nan")),
                dict(out_scale=float("inf")), dict(norm_weight=w[:1]), dict(norm_weight=w.int()), dict(norm_bias=b.cpu()),
                dict(norm_bias=b[:, :32])):
        with pytest.raises(ValueError):
            f(x, **bad)
    for bad in (x[0], x.half(), x.double(), x[:0], x[:, :, :0], torch.zeros(1, 1, 1, 257, device="cuda")):
        with pytest.raises(ValueError):
            f(bad)
    with pytest.raises(TypeError):
        f(x, norm_weight=3.0)
    with pytest.raises(TypeError):
        f(None)
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ValueError, match="forward-mode"):
            f(torch.autograd.forward_ad.make_dual(x, x))
    x.requires_grad_()
    y = f(x)
    torch.autograd.grad(y, x, dy)
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(y, x, dy)
    y = f(x)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(y, x, dy, create_graph=True)
