"""GPU tests of the norm and rotation of queries and keys (qk_norm_rotary, forward
and backward) and of appending to the paged cache, against float64."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _clean():
    da.get_device_error()
    yield
    assert da.get_device_error() == 0


def rows(g, dtype, B, H, T, D, layout="token"):
    x = torch.randn(B, T, H, D, generator=g).to(DT[dtype])
    if layout == "token":                       # a projection's output seen head-major
        return x.cuda().transpose(1, 2)
    if layout == "head":
        return x.transpose(1, 2).contiguous().cuda()
    if layout == "odd":                         # rows that start off 16-byte boundaries
        buf = torch.zeros(B, H, T, D + 3, dtype=DT[dtype], device="cuda")
        buf[..., 1:1 + D] = x.transpose(1, 2).cuda()
        return buf[..., 1:1 + D]
    assert layout == "strided"                  # not contiguous along the row
    return x.transpose(1, 2).cuda().repeat_interleave(2, -1)[..., ::2]


def d64(t):
    return None if t is None else t.detach().cpu().double()


def assert_within(got, want, bound, dtype, what):
    got = d64(got)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - (bound + ref.half_step(DT[dtype]) * want.abs() + 1e-30)
    assert over.max() <= 0, f"{what}: {over.max()} over the bound"


CASES = [  # dtype, B, H, Hk, T, D, R, layout
    ("bf16", 2, 3, 3, 17, 64, 64, "token"), ("bf16", 1, 4, 2, 300, 128, 128, "head"),
    ("bf16", 3, 2, 1, 5, 32, 16, "token"), ("bf16", 1, 1, 1, 1, 64, 64, "token"),
    ("bf16", 2, 2, 2, 9, 64, 32, "odd"), ("bf16", 2, 2, 2, 9, 64, 64, "strided"),
    ("bf16", 1, 3, 1, 33, 48, 24, "token"), ("bf16", 1, 2, 2, 7, 16, 8, "head"),
    ("bf16", 1, 2, 1, 40, 1, 0, "head"), ("bf16", 2, 40, 8, 65, 64, 0, "token"),
    ("f32", 2, 3, 3, 17, 64, 64, "token"), ("f32", 1, 4, 2, 100, 128, 64, "head"),
    ("f32", 2, 3, 1, 11, 16, 8, "token"), ("f32", 1, 2, 2, 13, 30, 10, "token"),
    ("f32", 1, 2, 2, 6, 32, 32, "odd"),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,weights", [("rms", "shared"), ("rms", "per_head"), ("rms", None), (None, None)])
def test_forward_and_backward(case, interleaved, norm, weights):
    dtype, B, H, Hk, T, D, R, layout = case
    g = torch.Generator().manual_seed(D * 1000 + T + R)
    xs = [rows(g, dtype, B, n, T, D, layout) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(5000, R, device="cuda") if R else (None, None)
    pos = torch.randint(0, 5000, (B, T), generator=g)
    qw = kw = None
    if weights:
        qw = (1 + 0.3 * torch.randn(*((H, D) if weights == "per_head" else (D,)), generator=g)).cuda()
        kw = (1 + 0.3 * torch.randn(*((Hk, D) if weights == "per_head" else (D,)), generator=g)).cuda()
    leaves = [x.detach().requires_grad_() for x in xs]
    ws = [w.requires_grad_() for w in (qw, kw) if w is not None]
    kw_args = dict(norm=norm, norm_eps=EPS, q_weight=qw, k_weight=kw, interleaved=interleaved)
    outs = da.qk_norm_rotary(*leaves, cos, sin, pos.cuda(), **kw_args)
    # the same without a graph, with int32 positions
    with torch.no_grad():
        plain = da.qk_norm_rotary(*xs, cos, sin, pos.cuda().int(), **kw_args)
    dys = [torch.randn(o.shape, generator=g).to(DT[dtype]).cuda() for o in outs]
    grads = torch.autograd.grad(outs, leaves + ws, dys)
    again = torch.autograd.grad(da.qk_norm_rotary(*leaves, cos, sin, pos.cuda(), **kw_args), leaves + ws, dys)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))       # no order of atomics
    dws = {}
    for i, (x, o, p, dy) in enumerate(zip(xs, outs, plain, dys)):
        w = (qw, kw)[i & 1]
        want, bound = ref.norm_rotate(d64(x), d64(w), d64(cos), d64(sin), pos, interleaved, norm, EPS)
        assert o.is_contiguous() and torch.equal(o, p)
        assert_within(o, want, bound, dtype, f"y{i}")
        dx, dw, size = ref.norm_rotate_backward(d64(x), d64(w), d64(cos), d64(sin), pos, interleaved, norm, EPS, d64(dy))
        # u by 3 roundings of |dy_a| + |dy_b| <= 2 max|dy|; with the norm r by (D/2 + 4),
        # the mean's sum of D products by D, and a few more, of terms no larger than
        # r (|w u| + |x| r |g x| r) <= 2 D r max|w u|
        d = d64(dy).abs().amax(-1, keepdim=True) * 2
        if norm:
            r = 1 / torch.sqrt((d64(x) ** 2).mean(-1, keepdim=True) + EPS)
            d = d * r * (d64(w).abs().max() if w is not None else 1.0) * 2 * (1.5 * D + 16)
        else:
            d = d * 3
        assert_within(grads[i], dx, ref.U * d, dtype, f"dx{i}")
        if w is not None:
            if i & 1 in dws:
                dw, size = dw + dws[i & 1][0], size + dws[i & 1][1]
            dws[i & 1] = (dw, size)
    for (i, (dw, size)), got in zip(sorted(dws.items()), grads[4:]):
        if weights == "shared":
            dw, size = dw.sum(0), size.sum(0)
        # a term is off by (D/2 + 10) u of twice its size at most (the pair's other part
        # may be the larger: counted by max over channels), a sum of N terms by N u
        n = 2 * B * T * (H, Hk)[i]
        tol = ref.U * ((2 * D + 40) * size.amax(-1, keepdim=True) + n * size)
        assert ((d64(got) - dw).abs() <= tol).all(), f"dw{i}"


@pytest.mark.parametrize("norm", ["rms", None])
def test_gradient_against_differences(norm):
    """Central differences of sum(y dy) along random directions, float32 rows."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(1, 2, 9, 64, generator=g).cuda()
    w = (1 + 0.3 * torch.randn(64, generator=g)).cuda() if norm else None
    cos, sin = da.rotary_tables(64, 64, device="cuda")
    dy = torch.randn(1, 2, 9, 64, generator=g).cuda()
    leaves = [x.clone().requires_grad_()] + ([w.clone().requires_grad_()] if norm else [])

    def f(x, w=None):
        y = da.qk_norm_rotary(x, None, None, None, cos, sin, norm=norm, q_weight=w)[0]
        return (y.double() * dy.double()).sum(), y

    grads = torch.autograd.grad(f(*leaves)[1], leaves, dy)
    for i, grad in enumerate(grads):
        v = torch.randn(leaves[i].shape, generator=g).cuda()
        step = 2.0 ** -7
        moved = [[t.detach() + (s * step * v if j == i else 0) for j, t in enumerate(leaves)] for s in (1, -1)]
        with torch.no_grad():
            diff = float((f(*moved[0])[0] - f(*moved[1])[0]) / (2 * step))
        want = float((grad.double() * v.double()).sum())
        # second-order remainder: step^2 times third derivatives of order |x|^-3 summed over
        # 1152 values of order 1 (norm only), and 2^-22 relative of each y over 2 step
        slack = 1152 ** 0.5 * 8 * (step * step if norm else 0) + 1152 ** 0.5 * 8 * 2.0 ** -22 / step
        assert abs(diff - want) <= slack, (diff, want, slack)


def test_shared_keys_and_left_out_tensors():
    g = torch.Generator().manual_seed(1)
    q, k = rows(g, "bf16", 2, 4, 10, 128), rows(g, "bf16", 2, 2, 10, 128)
    cos, sin = da.rotary_tables(10, 128, device="cuda")
    a = da.qk_norm_rotary(q, k, q, k, cos, sin)
    assert a[1] is a[3]
    b = da.qk_norm_rotary(q, None, None, k, cos, sin)
    assert b[1] is None and b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
    # the shared tensor's gradient is the sum of its two uses
    kl = k.detach().requires_grad_()
    _, k1, _, k2 = da.qk_norm_rotary(q, kl, q, kl, cos, sin)
    dy = torch.randn(k.shape, generator=g).to(torch.bfloat16).cuda()
    (g2,) = torch.autograd.grad(k1 + k2, kl, dy)
    (g1,) = torch.autograd.grad(da.qk_norm_rotary(None, kl, None, None, cos, sin)[1], kl, dy)
    assert torch.allclose(g2.float(), 2 * g1.float(), rtol=2.0 ** -7)
    # a gradient that never comes is zero
    ql = q.detach().requires_grad_()
    out = da.qk_norm_rotary(ql, kl, None, None, cos, sin)
    gq, gk = torch.autograd.grad(out[0].sum(), [ql, kl])
    assert torch.count_nonzero(gk) == 0 and torch.count_nonzero(gq) > 0


@pytest.mark.parametrize("D,H,Hk,T", [(64, 5, 3, 150), (128, 9, 2, 300), (48, 3, 2, 40)])
@pytest.mark.parametrize("q_heads", [True, False])
def test_a_weight_by_head_beside_a_shared_one(D, H, Hk, T, q_heads):
    """Q's weight by head and K's for all heads, and the reverse: each gradient is the one it
    has with both weights laid out its way."""
    g = torch.Generator().manual_seed(D + T)
    xs = [rows(g, "f32", 2, n, T, D) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(T, D, device="cuda")
    dys = [torch.randn(x.shape, generator=g).cuda() for x in xs]
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))

    def grads(q_by_head, k_by_head):
        a = (qw.expand(H, D) if q_by_head else qw).clone().requires_grad_()
        b = (kw.expand(Hk, D) if k_by_head else kw).clone().requires_grad_()
        out = da.qk_norm_rotary(*xs, cos, sin, q_weight=a, k_weight=b)
        return torch.autograd.grad(out, [a, b], dys)

    mixed = grads(q_heads, not q_heads)
    assert torch.equal(mixed[0], grads(q_heads, q_heads)[0])
    assert torch.equal(mixed[1], grads(not q_heads, not q_heads)[1])
    by_head, shared = grads(True, True), grads(False, False)
    for a, b, n in zip(by_head, shared, (H, Hk)):
        # the same terms in another order: N u of their sizes, about (4 B T n) half of |w x u|
        assert ((a.double().sum(0) - b.double()).abs() <= 2.0 ** -24 * 4 * T * n * 40).all()


@pytest.mark.parametrize("D,R", [(64, 64), (128, 64), (48, 24)])
@pytest.mark.parametrize("only", ["q", "k"])
@pytest.mark.parametrize("other", ["none", "fixed"])
def test_the_gradient_of_one_weight_alone(D, R, only, other):
    """One of the weights wants a gradient; the other is left out or wants none."""
    g = torch.Generator().manual_seed(D + R)
    B, H, Hk, T = 2, 3, 2, 12007                # several heads a block
    xs = [rows(g, "bf16", B, n, T, D) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(T, R, device="cuda")
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda().requires_grad_()
    fixed = (1 + 0.3 * torch.randn(D, generator=g)).cuda() if other == "fixed" else None
    weights = dict(q_weight=w, k_weight=fixed) if only == "q" else dict(q_weight=fixed, k_weight=w)
    outs = da.qk_norm_rotary(*xs, cos, sin, **weights, norm_eps=EPS)
    dys = [torch.randn(o.shape, generator=g).to(torch.bfloat16).cuda() for o in outs]
    dw, = torch.autograd.grad(outs, [w], dys)
    want, size, n = 0, 0, 0
    pos = torch.arange(T)[None].expand(B, T)
    for x, dy in list(zip(xs, dys))[0 if only == "q" else 1::2]:
        _, d, m = ref.norm_rotate_backward(d64(x), d64(w), d64(cos), d64(sin), pos, False, "rms", EPS, d64(dy))
        want, size, n = want + d.sum(0), size + m.sum(0), n + x.shape[0] * x.shape[1] * T
    tol = ref.U * ((2 * D + 40) * size.max() + n * size)
    assert ((d64(dw) - want).abs() <= tol).all()


def test_broadcast_rows_and_float16_weights():
    """A row tensor expanded over the batch (stride 0) and weights of another type."""
    g = torch.Generator().manual_seed(2)
    base = rows(g, "bf16", 1, 2, 6, 64, "head")
    leaf = base.detach().requires_grad_()
    w = torch.ones(64, dtype=torch.float16, device="cuda", requires_grad=True)
    cos, sin = da.rotary_tables(6, 64, device="cuda")
    y = da.qk_norm_rotary(leaf.expand(3, -1, -1, -1), None, None, None, cos, sin, q_weight=w)[0]
    assert y.shape == (3, 2, 6, 64) and torch.equal(y[0], y[2])
    gx, gw = torch.autograd.grad(y, [leaf, w], torch.ones_like(y))
    assert gx.shape == leaf.shape and gw.dtype == torch.float16
    one = da.qk_norm_rotary(leaf, None, None, None, cos, sin, q_weight=w)[0]
    (g1,) = torch.autograd.grad(one, [leaf], torch.ones_like(one))
    assert torch.allclose(gx.float(), 3 * g1.float(), rtol=2.0 ** -6, atol=1e-2)


@pytest.mark.parametrize("D,R", [(64, 64), (48, 24)])
def test_positions_outside_the_tables(D, R):
    g = torch.Generator().manual_seed(3)
    x = rows(g, "bf16", 1, 2, 8, D)
    cos, sin = da.rotary_tables(100, R, device="cuda")
    pos = torch.tensor([0, 99, 100, -1, 5, 2 ** 40, -2 ** 40, 7], device="cuda")
    y = da.qk_norm_rotary(x, None, None, None, cos, sin, pos)[0]
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    bad = torch.tensor([0, 0, 1, 1, 0, 1, 1, 0], dtype=torch.bool)
    assert torch.isnan(y[:, :, bad]).all() and torch.isfinite(y[:, :, ~bad]).all()
    xl = x.detach().requires_grad_()
    w = torch.ones(D, device="cuda")
    out = da.qk_norm_rotary(xl, None, None, None, cos, sin, pos, q_weight=w)[0]
    (dx,) = torch.autograd.grad(out, xl, torch.ones_like(out))
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    assert torch.isnan(dx[:, :, bad]).all() and torch.isfinite(dx[:, :, ~bad]).all()


def test_capture_and_other_streams():
    """Forward and backward captured into a graph and replayed on new inputs; a call on a
    side stream."""
    g = torch.Generator().manual_seed(4)
    x = rows(g, "bf16", 2, 4, 50, 64, "head")
    w = torch.ones(64, device="cuda")
    cos, sin = da.rotary_tables(50, 64, device="cuda")
    dy = torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda()
    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()

    def step():
        y = da.qk_norm_rotary(xl, None, None, None, cos, sin, q_weight=wl)[0]
        return (y, *torch.autograd.grad(y, [xl, wl], dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    new = torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda()
    with torch.no_grad():
        xl.copy_(new)
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert not torch.equal(first[0], held[0])


def test_captured_backward_beside_a_living_graph():
    """Gradients added in a capture to leaves that an eager graph holds: refused where that
    graph was made on the default stream, right where it was made on another."""
    g = torch.Generator().manual_seed(9)
    x = rows(g, "bf16", 2, 4, 50, 64, "head")
    cos, sin = da.rotary_tables(50, 64, device="cuda")
    dy = torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda()
    for where in ("default", "side"):
        leaf = x.clone().requires_grad_()
        w = torch.ones(64, device="cuda").requires_grad_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side if where == "side" else torch.cuda.default_stream()):
            eager = da.qk_norm_rotary(leaf * 1, None, None, None, cos, sin, q_weight=w)[0]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()

        def captured():
            with torch.cuda.graph(graph, stream=side if where == "side" else None):
                da.qk_norm_rotary(leaf * 1, None, None, None, cos, sin, q_weight=w)[0].backward(dy)

        if where == "default":
            with pytest.raises(RuntimeError, match="default stream"):
                captured()
            assert leaf.grad is None and w.grad is None
            continue
        captured()
        graph.replay()
        want = torch.autograd.grad(eager, [leaf, w], dy)
        torch.cuda.synchronize()
        assert torch.equal(leaf.grad, want[0]) and torch.equal(w.grad, want[1])


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPEND = [  # dtype, Hk, T, D, Dv, R, page, layout
    ("bf16", 2, 1, 64, 128, 64, 64, "token"), ("bf16", 3, 37, 128, 128, 64, 16, "token"),
    ("bf16", 1, 5, 32, 64, 32, 1, "head"), ("bf16", 2, 9, 48, 30, 24, 7, "token"),
    ("bf16", 2, 9, 64, 128, 0, 16, "odd"), ("f32", 2, 20, 64, 128, 64, 32, "token"),
    ("f32", 1, 3, 10, 256, 4, 5, "head"),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("norm", [None, "rms"])
def test_append(case, shared, norm):
    dtype, Hk, T, D, Dv, R, page, layout = case
    g = torch.Generator().manual_seed(T + D)
    lens = [0, 1, page, 3 * page - 1, 2 * page + 3]
    new = [T, max(T - 1, 0), 0, T, min(T, 3)]
    B = len(lens)
    per = max(-(-(n + T) // page) for n in lens)
    pool = B * per + 2
    order = torch.randperm(pool, generator=g)[:B * per].reshape(B, per).int()
    k1, k2, v = (rows(g, dtype, B, Hk, T, n, layout) for n in (D, D, Dv))
    caches = [torch.randn(pool, Hk, page, n, generator=g).to(DT[dtype]).cuda() for n in (D, D, Dv)]
    if layout == "token":                       # a cache stored [pages, page, heads, width]
        caches = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in caches]
    before = [c.clone() for c in caches]
    cos, sin = da.rotary_tables(4 * page + 2 * T + 8, R, device="cuda") if R else (None, None)
    kw = (1 + 0.3 * torch.randn(Hk, D, generator=g)).cuda() if norm else None
    pos = torch.randint(0, 4 * page, (B, T), generator=g) if shared else None     # or the index itself
    da.paged_cache_append(k1, k1 if shared else k2, v, caches[0], caches[0] if shared else caches[1], caches[2],
                          order.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                          torch.tensor(new, dtype=torch.int32).cuda(), cos, sin,
                          None if pos is None else pos.cuda(), norm=norm, norm_eps=EPS, k_weight=kw)
    at = torch.tensor(lens)[:, None] + torch.arange(T)
    for x, cache, old, w in ((k1, caches[0], before[0], kw), (k2, caches[1], before[1], kw), (v, caches[2], before[2], None)):
        if x is k2 and shared:
            assert torch.equal(cache, old)
            continue
        if x is v:
            want, bound = d64(x), torch.zeros(x.shape, dtype=torch.float64)
        else:
            want, bound = ref.norm_rotate(d64(x), d64(w), d64(cos), d64(sin), at if pos is None else pos, False, norm, EPS)
        untouched = torch.ones(pool, page, dtype=torch.bool)
        for b in range(B):
            for t in range(new[b]):
                pg, slot = int(order[b, int(at[b, t]) // page]), int(at[b, t]) % page
                untouched[pg, slot] = False
                assert_within(cache[pg, :, slot], want[b, :, t], bound[b, :, t], dtype, f"b={b} t={t}")
                if x is v:
                    assert torch.equal(cache[pg, :, slot], x[b, :, t])
        keep = untouched[:, None, :, None].expand(cache.shape)
        assert torch.equal(cache.cpu()[keep], old.cpu()[keep])


def test_append_out_of_range():
    """Tokens past the table, on pages outside the cache and at positions outside the
    tables are left out, and nothing else changes."""
    g = torch.Generator().manual_seed(9)
    page, B, T = 16, 4, 3
    k, v = rows(g, "bf16", B, 2, T, 64), rows(g, "bf16", B, 2, T, 128)
    kc = torch.zeros(6, 2, page, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(6, 2, page, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 6], [-1, 3], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([31, 15, -1, 0], dtype=torch.int32, device="cuda")   # 2 past the end, 2 on page 6, 1 below 0 and 2 on page -1
    cos, sin = da.rotary_tables(2 * page, 64, device="cuda")
    da.paged_cache_append(k, k, v, kc, kc, vc, table, lens, None, cos, sin)
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    written = {(1, 15): (0, 0), (2, 15): (1, 0), (4, 0): (3, 0), (4, 1): (3, 1), (4, 2): (3, 2)}
    for pg in range(6):
        for s in range(page):
            if (pg, s) in written:
                b, t = written[pg, s]
                assert torch.equal(vc[pg, :, s], v[b, :, t]) and torch.count_nonzero(kc[pg, :, s]) > 0
            else:
                assert torch.count_nonzero(vc[pg, :, s]) == 0 and torch.count_nonzero(kc[pg, :, s]) == 0


def test_large_offsets():
    """A cache of more than 2^31 elements: the last page is written where it belongs."""
    pages, page, Hk = 9000, 128, 16
    kc = torch.zeros(pages, Hk, page, 128, dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 31
    k = torch.randn(1, Hk, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    da.paged_cache_append(k, k, k, kc, kc, kc.clone(), table, torch.tensor([126], dtype=torch.int32, device="cuda"))
    assert torch.equal(kc[-1, :, 126:], k[0]) and torch.count_nonzero(kc[-1, :, :126]) == 0
    assert torch.count_nonzero(kc[:-1].view(torch.int16)) == 0


def test_more_than_2_31_elements():
    """Rows whose elements lie past 2^31, with gradients: the first and last tokens'."""
    T, H, D = (1 << 23) + 37, 2, 128
    assert T * H * D > 2 ** 31
    g = torch.Generator().manual_seed(5)
    x = torch.zeros(1, T, H, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    dy = torch.zeros_like(x)
    ends = torch.cat([torch.arange(5), torch.arange(T - 40, T)])
    some, up = (torch.randn(1, H, len(ends), D, generator=g).to(torch.bfloat16) for _ in range(2))
    x[:, :, ends.cuda()], dy[:, :, ends.cuda()] = some.cuda(), up.cuda()
    cos, sin = da.rotary_tables(64, D)
    pos = (torch.arange(T) % 64).int()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda().requires_grad_()
    x.requires_grad_()
    y = da.qk_norm_rotary(x, None, None, None, cos.cuda(), sin.cuda(), pos.cuda(), q_weight=w)[0]
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    args = (some.double(), d64(w), cos.double(), sin.double(), pos[ends].long()[None], False, "rms", EPS)
    want, bound = ref.norm_rotate(*args)
    assert_within(y[:, :, ends.cuda()].detach(), want, bound, "bf16", "y")
    want, want_dw, size = ref.norm_rotate_backward(*args, up.double())
    # bounds as in test_forward_and_backward
    r = 1 / torch.sqrt((some.double() ** 2).mean(-1, keepdim=True) + EPS)
    d = up.double().abs().amax(-1, keepdim=True) * 4 * r * d64(w).abs().max() * (1.5 * D + 16)
    assert_within(dx[:, :, ends.cuda()], want, ref.U * d, "bf16", "dx")
    want_dw, size = want_dw.sum(0), size.sum(0)
    tol = ref.U * ((2 * D + 40) * size.max() + H * len(ends) * size)
    assert ((d64(dw) - want_dw).abs() <= tol).all()
    assert not dx[:, :, 5:T - 40].any()
