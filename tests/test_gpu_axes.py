"""GPU tests of positions with several axes (qk_norm_rotary and paged_cache_append with
sections), and of a whole cross-attention block: rotation, attention, norm.

A rotation by several axes is the rotation by one, with a table row of its own for every
token, put together from its axes' rows: tests/paged_reference.py and its bounds are used
with those rows."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import block_reference, paged_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


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


def rows(g, dtype, B, H, T, D, odd=False):
    x = torch.randn(B, T, H, D, generator=g).to(dtype)
    if odd:
        buf = torch.zeros(B, H, T, D + 3, dtype=dtype, device="cuda")
        buf[..., 1:1 + D] = x.transpose(1, 2).cuda()
        return buf[..., 1:1 + D]
    return x.cuda().transpose(1, 2)


def gathered(cos, sin, pos, sections):
    """Tables [B T, R/2] of each token's own rows, and positions into them."""
    B, T, _ = pos.shape
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)])
    pair = torch.arange(len(axis))
    at = pos[:, :, axis].reshape(B * T, -1)
    return d64(cos)[at, pair], d64(sin)[at, pair], torch.arange(B * T).reshape(B, T)


def within(got, want, bound, dtype, what):
    got = d64(got)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - (bound + ref.half_step(dtype) * want.abs() + 1e-30)
    assert over.max() <= 0, f"{what}: {over.max()} over the bound"


CASES = [  # dtype, B, H, Hk, T, D, R, sections, odd rows
    (BF, 2, 3, 3, 17, 64, 64, (8, 12, 12), False), (BF, 1, 4, 2, 300, 128, 128, (16, 24, 24), False),
    (BF, 2, 2, 1, 9, 64, 64, (32,), False), (BF, 2, 2, 2, 9, 64, 32, (4, 4, 4, 4), False),
    (BF, 1, 2, 2, 33, 64, 64, (3, 13, 16), False), (BF, 1, 2, 2, 9, 64, 64, (16, 16), True),
    (BF, 2, 2, 1, 21, 48, 24, (5, 7), False), (BF, 1, 1, 1, 1, 64, 64, (1, 31), False),
    (F32, 2, 3, 3, 17, 64, 64, (8, 12, 12), False), (F32, 1, 4, 2, 100, 128, 64, (8, 8, 16), False),
    (F32, 2, 2, 1, 11, 32, 32, (4, 12), False), (F32, 1, 2, 2, 13, 30, 10, (2, 3), False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,weights", [("rms", "shared"), ("rms", "per_head"), (None, None)])
def test_forward_and_backward(case, interleaved, norm, weights):
    dtype, B, H, Hk, T, D, R, sections, odd = case
    g = torch.Generator().manual_seed(D * 1000 + T + R)
    xs = [rows(g, dtype, B, n, T, D, odd) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(500, R, device="cuda", sections=sections)
    pos = torch.randint(0, 500, (B, T, len(sections)), generator=g)
    qw = kw = None
    if weights:
        qw = (1 + 0.3 * torch.randn(*((H, D) if weights == "per_head" else (D,)), generator=g)).cuda()
        kw = (1 + 0.3 * torch.randn(*((Hk, D) if weights == "per_head" else (D,)), generator=g)).cuda()
    leaves = [x.detach().requires_grad_() for x in xs]
    ws = [w.requires_grad_() for w in (qw, kw) if w is not None]
    args = dict(norm=norm, norm_eps=EPS, q_weight=qw, k_weight=kw, interleaved=interleaved, sections=sections)
    outs = da.qk_norm_rotary(*leaves, cos, sin, pos.cuda(), **args)
    # int32 positions, axes before tokens in memory, and a list of sections
    turned = pos.permute(2, 0, 1).contiguous().int().cuda().permute(1, 2, 0)
    with torch.no_grad():
        plain = da.qk_norm_rotary(*xs, cos, sin, turned, **{**args, "sections": list(sections)})
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    dys = [torch.randn(o.shape, generator=g).to(dtype).cuda() for o in outs]
    grads = torch.autograd.grad(outs, leaves + ws, dys)
    c, s, p = gathered(cos, sin, pos, sections)
    dws = {}
    for i, (x, o, dy) in enumerate(zip(xs, outs, dys)):
        w = (qw, kw)[i & 1]
        want, bound = ref.norm_rotate(d64(x), d64(w), c, s, p, interleaved, norm, EPS)
        within(o, want, bound, dtype, f"y{i}")
        dx, dw, size = ref.norm_rotate_backward(d64(x), d64(w), c, s, p, interleaved, norm, EPS, d64(dy))
        # as the bounds of one axis: u by 3 roundings of 2 max|dy|, with the norm (1.5 D + 16) of
        # terms no larger than 2 r max|w u|
        d = d64(dy).abs().amax(-1, keepdim=True) * 2
        if norm:
            r = 1 / torch.sqrt((d64(x) ** 2).mean(-1, keepdim=True) + EPS)
            d = d * r * (d64(w).abs().max() if w is not None else 1.0) * 2 * (1.5 * D + 16)
        else:
            d = d * 3
        within(grads[i], dx, ref.U * d, dtype, f"dx{i}")
        if w is not None:
            if i & 1 in dws:
                dw, size = dw + dws[i & 1][0], size + dws[i & 1][1]
            dws[i & 1] = (dw, size)
    for (i, (dw, size)), got in zip(sorted(dws.items()), grads[4:]):
        if weights == "shared":
            dw, size = dw.sum(0), size.sum(0)
        n = 2 * B * T * (H, Hk)[i]
        tol = ref.U * ((2 * D + 40) * size.amax(-1, keepdim=True) + n * size)
        assert ((d64(got) - dw).abs() <= tol).all(), f"dw{i}"


def test_equal_positions_are_one_position():
    """Text tokens have the same position on every axis: the rotation of one axis, with the same
    table; and one section is the rotation without sections, bit for bit."""
    g = torch.Generator().manual_seed(1)
    cos, sin = da.rotary_tables(100, 64, device="cuda")
    pos = torch.randint(0, 100, (2, 40), generator=g).cuda()
    for dtype in (BF, F32):
        x = rows(g, dtype, 2, 4, 40, 64)
        want = da.qk_norm_rotary(x, None, None, None, cos, sin, pos)[0]
        for sections in ((32,), (8, 12, 12)):
            got = da.qk_norm_rotary(x, None, None, None, cos, sin, pos[:, :, None].expand(-1, -1, len(sections)), sections=sections)[0]
            assert torch.equal(got, want)
    flat = da.qk_norm_rotary(x, None, None, None, cos, sin, pos[0][:, None].expand(-1, 2), sections=(16, 16))[0]
    assert torch.equal(flat, da.qk_norm_rotary(x, None, None, None, cos, sin, pos[0])[0])


@pytest.mark.parametrize("D,sections", [(64, (8, 12, 12)), (64, (3, 29))])
def test_positions_outside_the_tables(D, sections):
    """A token with any position outside: rows of NaN, gradients too, and it is reported."""
    g = torch.Generator().manual_seed(2)
    x = rows(g, BF, 1, 2, 12, D).requires_grad_()
    cos, sin = da.rotary_tables(50, D, device="cuda", sections=sections)
    pos = torch.randint(0, 50, (12, len(sections)), generator=g)
    pos[3, 0], pos[7, -1] = 50, -1
    y = da.qk_norm_rotary(x, None, None, None, cos, sin, pos.cuda(), sections=sections)[0]
    dx, = torch.autograd.grad(y, x, torch.ones_like(y))
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    bad = torch.zeros(12, dtype=torch.bool)
    bad[[3, 7]] = True
    for t in (y, dx):
        assert t[:, :, bad].isnan().all() and t[:, :, ~bad].isfinite().all()


@pytest.mark.parametrize("dtype,D,Dv,sections", [(BF, 64, 128, (8, 12, 12)), (F32, 32, 64, (4, 12)), (BF, 48, 30, (5, 7))])
@pytest.mark.parametrize("shared", [False, True])
def test_append(dtype, D, Dv, sections, shared):
    g = torch.Generator().manual_seed(D)
    page, T, Hk, lens, new = 16, 7, 2, [0, 16, 41, 30], [7, 6, 0, 7]
    B, per = 4, 4
    order = torch.randperm(B * per + 1, generator=g)[:B * per].reshape(B, per).int()
    k1, k2, v = (rows(g, dtype, B, Hk, T, n) for n in (D, D, Dv))
    caches = [torch.randn(B * per + 1, Hk, page, n, generator=g).to(dtype).cuda() for n in (D, D, Dv)]
    before = [c.clone() for c in caches]
    cos, sin = da.rotary_tables(200, 2 * sum(sections), device="cuda", sections=sections)
    pos = torch.randint(0, 200, (B, T, len(sections)), generator=g)
    pos[1, 2, 1] = 200                          # out of the table: not written
    w = (1 + 0.3 * torch.randn(Hk, D, generator=g)).cuda()
    da.paged_cache_append(k1, k1 if shared else k2, v, caches[0], caches[0] if shared else caches[1], caches[2], order.cuda(),
                          torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(new, dtype=torch.int32).cuda(), cos, sin,
                          pos.cuda(), norm="rms", norm_eps=EPS, k_weight=w, sections=sections)
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    pos[1, 2, 1] = 0
    c, s, p = gathered(cos, sin, pos, sections)
    for x, cache, old in ((k1, caches[0], before[0]), (k2, caches[1], before[1]), (v, caches[2], before[2])):
        expect = old.clone()
        if x is k2 and shared:
            assert torch.equal(cache, old)
            continue
        want, bound = (d64(x), torch.zeros(1)) if x is v else ref.norm_rotate(d64(x), d64(w), c, s, p, False, "rms", EPS)
        for b in range(B):
            for t in range(new[b]):
                if (b, t) == (1, 2):
                    continue
                pg, slot = int(order[b, (lens[b] + t) // page]), (lens[b] + t) % page
                within(cache[pg, :, slot], want[b, :, t], bound if x is v else bound[b, :, t], dtype, f"b={b} t={t}")
                expect[pg, :, slot] = cache[pg, :, slot]
        assert torch.equal(cache, expect)


def test_append_is_the_rotation():
    """Keys appended to a cache equal those that qk_norm_rotary gives, bit for bit."""
    g = torch.Generator().manual_seed(5)
    sections = (16, 24, 24)
    k, v = rows(g, BF, 2, 8, 33, 128), rows(g, BF, 2, 8, 33, 128)
    cos, sin = da.rotary_tables(64, 128, device="cuda")
    pos = torch.randint(0, 64, (2, 33, 3), generator=g).cuda()
    cache, vc = (torch.zeros(2, 8, 64, 128, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    da.paged_cache_append(k, k, v, cache, cache, vc, table, torch.tensor([5, 31], dtype=torch.int32, device="cuda"), None, cos, sin, pos,
                          norm="rms", norm_eps=EPS, sections=sections)
    want = da.qk_norm_rotary(None, k, None, None, cos, sin, pos, norm_eps=EPS, sections=sections)[1]
    assert torch.equal(cache[1, :, 5:38], want[0]) and torch.equal(cache[0, :, 31:64], want[1])
    assert torch.equal(vc[1, :, 5:38], v[0])


def test_captured_and_replayed():
    """Forward and backward in a graph follow new positions."""
    g = torch.Generator().manual_seed(6)
    x = rows(g, BF, 2, 4, 50, 64).requires_grad_()
    cos, sin = da.rotary_tables(64, 64, device="cuda", sections=(8, 12, 12))
    pos = torch.randint(0, 64, (2, 50, 3), generator=g).cuda()
    dy = torch.randn(2, 4, 50, 64, generator=g).to(BF).cuda()

    def step():
        y = da.qk_norm_rotary(x, None, None, None, cos, sin, pos, sections=(8, 12, 12))[0]
        return y.detach(), torch.autograd.grad(y, x, dy)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    pos.copy_(torch.randint(0, 64, (2, 50, 3), generator=g))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals():
    g = torch.Generator().manual_seed(7)
    x = rows(g, BF, 1, 2, 5, 64)
    cos, sin = da.rotary_tables(20, 64, device="cuda")
    pos = torch.zeros(1, 5, 2, dtype=torch.int32, device="cuda")

    def f(sections, pos=pos, cos=cos, sin=sin):
        return da.qk_norm_rotary(x, None, None, None, cos, sin, pos, sections=sections)
    f((16, 16))
    for bad in ((), (16,), (16, 17), (32, 0), (-1, 33), (8, 8, 16), (8, 8, 8, 4, 4), (10 ** 30, 1)):
        with pytest.raises(ValueError):
            f(bad)
    for bad in ("16", 32, (16.0, 16.0), (None, 32), torch.tensor([16, 16])):
        with pytest.raises(TypeError):
            f(bad)
    for bad in (None, pos[0, :, 0], pos[:, :4], pos.cpu(), pos.float(), pos.expand(2, -1, -1), pos[..., None]):
        with pytest.raises((ValueError, TypeError)):
            f((16, 16), pos=bad)
    with pytest.raises(ValueError):
        f((16, 16), cos=None, sin=None)
    c, v = torch.zeros(1, 2, 16, 64, dtype=BF, device="cuda"), torch.zeros(1, 2, 16, 64, dtype=BF, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        da.paged_cache_append(x, x, x, c, c, v, table, lens, cos=cos, sin=sin, sections=(16, 16))


# ------------------------------------------------------------------ the operators together
def block(q1, k1, q2, v, qw, kw, nw, nb, lam, cos, sin, qpos, kpos, sections, lens):
    """Rotate, attend over the states, norm each head: what a layer does between projections."""
    a, _, b, _ = da.qk_norm_rotary(q1, None, q2, None, cos, sin, qpos, q_weight=qw, norm_eps=EPS, sections=sections)
    _, k, _, _ = da.qk_norm_rotary(None, k1, None, None, cos, sin, kpos, k_weight=kw, norm_eps=EPS, sections=sections)
    o = da.differential_cross_attention(a, k, b, k, v, lam, kv_lengths=lens)
    return da.differential_head_norm(o, "group", EPS, nw, nb, 0.2)


def test_a_block_in_training():
    """float32, against autograd of the same formulas in float64: the gradients of every input and
    parameter; the bounds go by the tensors' norms.  Each step is off by some 100 U of its result's
    size at most (the operators' own tests bound it elementwise) and passes on what came before
    with a gain that softmax, norms and products of this size keep below 100."""
    g = torch.Generator().manual_seed(8)
    B, H, Hk, Tq, Tk, D, sections, lens = 2, 4, 2, 50, 70, 64, (8, 12, 12), [70, 33]
    cos, sin = da.rotary_tables(100, D, sections=sections)
    qpos, kpos = torch.randint(0, 100, (B, Tq, 3), generator=g), torch.randint(0, 100, (Tk, 3), generator=g)
    ts = [torch.randn(B, H, Tq, D, generator=g), torch.randn(B, Hk, Tk, D, generator=g), torch.randn(B, H, Tq, D, generator=g),
          torch.randn(B, Hk, Tk, 128, generator=g), 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(Hk, D, generator=g),
          1 + 0.2 * torch.randn(H, 128, generator=g), 0.2 * torch.randn(H, 128, generator=g), torch.tensor(0.8)]
    dy = torch.randn(B, H, Tq, 128, generator=g)
    own = [t.cuda().requires_grad_() for t in ts]
    y = block(*own, cos.cuda(), sin.cuda(), qpos.cuda(), kpos.cuda(), sections, torch.tensor(lens, dtype=torch.int32).cuda())
    grads = torch.autograd.grad(y, own, dy.cuda())

    q1, k1, q2, v, qw, kw, nw, nb, lam = (t.double().requires_grad_() for t in ts)
    c, s, p = gathered(cos, sin, qpos, sections)
    kc, ks, kp = gathered(cos, sin, kpos[None].expand(B, -1, -1), sections)

    def turn(x, w, c, s, p):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (w if w.dim() == 1 else w[None, :, None])
        h = c.shape[1]
        c, s = c[p][:, None], s[p][:, None]
        return torch.cat([n[..., :h] * c - n[..., h:] * s, n[..., h:] * c + n[..., :h] * s], -1)

    a, b, k = turn(q1, qw, c, s, p), turn(q2, qw, c, s, p), turn(k1, kw, kc, ks, kp)
    seen = torch.arange(Tk) < torch.tensor(lens)[:, None]
    A = [torch.softmax((q @ k.repeat_interleave(2, 1).transpose(-1, -2) / 8).masked_fill(~seen[:, None, None], -float("inf")), -1) for q in (a, b)]
    o = (A[0] - lam * A[1]) @ v.repeat_interleave(2, 1)
    o = o - o.mean(-1, keepdim=True)
    want = 0.2 * (o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * nw[:, None] + nb[:, None])
    leaves = [q1, k1, q2, v, qw, kw, nw, nb, lam]
    wants = torch.autograd.grad(want, leaves, dy.double())
    for got, w in zip((y, *grads), (want, *wants)):
        assert (d64(got) - w.detach()).norm() <= 1e4 * block_reference.U * w.norm()


@pytest.mark.parametrize("D,Hk", [(64, 4), (128, 2)])
def test_a_block_in_bf16_and_token_by_token(D, Hk):
    """The same block in bf16: a captured training step repeats the eager one's bits, and serving the
    rows one at a time through the fused epilogue agrees with the whole sequence's to the roundings
    of O to bf16 that the fused form leaves out."""
    g = torch.Generator().manual_seed(9)
    B, H, Tq, Tk = 2, 4, 9, 130
    sections, lens = (D // 8, D // 8, D // 4), torch.tensor([130, 64], dtype=torch.int32, device="cuda")
    cos, sin = da.rotary_tables(200, D, device="cuda", sections=sections)
    qpos, kpos = torch.randint(0, 200, (B, Tq, 3), generator=g).cuda(), torch.randint(0, 200, (Tk, 3), generator=g).cuda()
    q1, q2 = (rows(g, BF, B, H, Tq, D).requires_grad_() for _ in range(2))
    k1, v = rows(g, BF, B, Hk, Tk, D).requires_grad_(), rows(g, BF, B, Hk, Tk, 128).requires_grad_()
    nw = (1 + 0.2 * torch.randn(H, 128, generator=g)).cuda().requires_grad_()
    lam = torch.tensor(0.8, device="cuda")
    dy = torch.randn(B, H, Tq, 128, generator=g).to(BF).cuda()
    leaves = [q1, k1, q2, v, nw]

    def step():
        y = block(q1, k1, q2, v, None, None, nw, None, lam, cos, sin, qpos, kpos, sections, lens)
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, held))
    with torch.no_grad():
        _, k, _, _ = da.qk_norm_rotary(None, k1, None, None, cos, sin, kpos, norm_eps=EPS, sections=sections)
        for t in range(Tq):
            a, _, b, _ = da.qk_norm_rotary(q1[:, :, t:t + 1], None, q2[:, :, t:t + 1], None, cos, sin, qpos[:, t:t + 1], norm_eps=EPS, sections=sections)
            y = da.differential_cross_attention(a, k, b, k, v, lam, lens, norm="group", norm_eps=EPS, norm_weight=nw.detach(), out_scale=0.2)
            want = eager[0][:, :, t:t + 1].double()
            # both forms' weights and results are rounded to bf16 (2^-8 of sums of |terms|): by norms
            assert (y.double() - want).norm() <= 4 * 2.0 ** -8 * want.norm()
