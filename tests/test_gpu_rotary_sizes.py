"""GPU tests of qk_norm_rotary and paged_cache_append at sizes where a block takes several
heads, against float64 at some of the tokens; and of the weights' gradients where nothing
cancels in them, so that a head, a tensor or a run of tokens that is left out shows."""
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


def rows(g, dtype, B, H, T, D):
    return torch.randn(B, T, H, D, generator=g, device="cuda").to(DT[dtype]).transpose(1, 2)


def d64(t):
    return None if t is None else t.detach().cpu().double()


def assert_within(got, want, bound, dtype, what):
    got = d64(got)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - (bound + ref.half_step(DT[dtype]) * want.abs() + 1e-30)
    assert over.max() <= 0, f"{what}: {over.max()} over the bound"


def heads_per_block(dtype, D, tokens, heads):
    """As csrc/rotary.cu has it, to see that the sizes below are what they are for."""
    lanes = D // (16 if dtype == "bf16" else 8)
    want = -(-tokens * lanes // 256) * heads // (8 * torch.cuda.get_device_properties(0).multi_processor_count)
    return max(1, want) if want < 4 else min(16, want // 4 * 4)


# dtype, D, R, H, Hk, T, heads a block: whole batches of four heads and not, more than one of them,
# heads that the last block of a tensor has fewer of
SIZES = [("bf16", 128, 128, 19, 5, 1700, 2), ("bf16", 128, 64, 19, 5, 4800, 4), ("bf16", 64, 64, 19, 3, 16000, 8),
         ("bf16", 128, 128, 19, 5, 14000, 16), ("f32", 128, 128, 19, 5, 1600, 3), ("f32", 64, 32, 17, 6, 7000, 8)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,per_head", [("rms", True), ("rms", False), (None, False)])
def test_several_heads_a_block(size, interleaved, norm, per_head):
    dtype, D, R, H, Hk, T, hpb = size
    assert heads_per_block(dtype, D, T, 2 * (H + Hk)) == hpb
    g = torch.Generator("cuda").manual_seed(T)
    xs = [rows(g, dtype, 1, n, T, D) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(4096, R, device="cuda")
    pos = torch.randint(0, 4096, (1, T), generator=g, device="cuda")
    qw, kw = ((1 + 0.3 * torch.randn(*((n, D) if per_head else (D,)), generator=g, device="cuda")) if norm else None
              for n in (H, Hk))
    leaves = [x.detach().requires_grad_() for x in xs]
    outs = da.qk_norm_rotary(*leaves, cos, sin, pos, norm=norm, norm_eps=EPS, q_weight=qw, k_weight=kw,
                             interleaved=interleaved)
    dys = [torch.randn(o.shape, generator=g, device="cuda").to(DT[dtype]) for o in outs]
    grads = torch.autograd.grad(outs, leaves, dys)
    at = torch.cat([torch.arange(3), torch.randint(0, T, (40,)), torch.arange(T - 3, T)]).cuda()
    for i, (x, o, dx, dy) in enumerate(zip(xs, outs, grads, dys)):
        w = (qw, kw)[i & 1]
        args = (d64(x[:, :, at]), d64(w), d64(cos), d64(sin), pos[:, at].cpu(), interleaved, norm, EPS)
        want, bound = ref.norm_rotate(*args)
        assert_within(o[:, :, at], want, bound, dtype, f"y{i}")
        want, _, _ = ref.norm_rotate_backward(*args, d64(dy[:, :, at]))
        # u by 3 roundings of |dy_a| + |dy_b| <= 2 max|dy|; with the norm r by (D/2 + 4), the mean's
        # sum of D products by D, and a few more, of terms no larger than 2 D r max|w u|
        d = d64(dy[:, :, at]).abs().amax(-1, keepdim=True) * 2
        if norm:
            r = 1 / torch.sqrt((args[0] ** 2).mean(-1, keepdim=True) + EPS)
            d = d * r * d64(w).abs().max() * 2 * (1.5 * D + 16)
        else:
            d = d * 3
        assert_within(dx[:, :, at], want, ref.U * d, dtype, f"dx{i}")


@pytest.mark.parametrize("dtype,D,Dv,Hk,T,hpb", [("bf16", 128, 256, 19, 1700, 2), ("bf16", 128, 256, 19, 3100, 4),
                                                 ("bf16", 64, 128, 19, 11000, 8), ("f32", 128, 128, 19, 5500, 16)])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_append_of_several_heads_a_block(dtype, D, Dv, Hk, T, hpb, layout):
    assert heads_per_block(dtype, D, T, 3 * Hk) == hpb
    g = torch.Generator("cuda").manual_seed(T)
    page, before = 64, 37
    pages = -(-(T + before) // page)
    k1, k2, v = (rows(g, dtype, 1, Hk, T, n) for n in (D, D, Dv))
    caches = [torch.zeros(pages + 2, *((Hk, page) if layout == "head" else (page, Hk)), n, dtype=DT[dtype], device="cuda")
              for n in (D, D, Dv)]
    if layout == "token":
        caches = [c.transpose(1, 2) for c in caches]
    order = torch.randperm(pages + 2, generator=g, device="cuda")[:pages].int()
    cos, sin = da.rotary_tables(T + before, D, device="cuda")
    kw = 1 + 0.3 * torch.randn(Hk, D, generator=g, device="cuda")
    da.paged_cache_append(k1, k2, v, *caches, order[None], torch.full((1,), before, dtype=torch.int32, device="cuda"), None,
                          cos, sin, norm="rms", norm_eps=EPS, k_weight=kw)
    # every row where it belongs: the values bit for bit, and of the keys some to the bound
    index = torch.arange(T, device="cuda") + before
    pg, slot = order[index // page].long(), index % page
    assert torch.equal(caches[2][pg, :, slot], v[0].transpose(0, 1))
    at = torch.cat([torch.arange(3), torch.randint(0, T, (60,)), torch.arange(T - 3, T)]).cuda()
    for x, cache in ((k1, caches[0]), (k2, caches[1])):
        want, bound = ref.norm_rotate(d64(x[:, :, at]), d64(kw), d64(cos), d64(sin), index[at].cpu()[None], False, "rms", EPS)
        assert_within(cache[pg[at], :, slot[at]].transpose(0, 1)[None], want, bound, dtype, "keys")
        # no other slot
        kept = torch.ones(pages + 2, page, dtype=torch.bool, device="cuda")
        kept[pg, slot] = False
        assert torch.count_nonzero(cache.transpose(1, 2)[kept]) == 0
        assert (cache.transpose(1, 2)[~kept].abs().amax(-1) > 0).all()


# Sums of squares.  dy is the rotation of x, so that u = x (but for dy's rounding) and every term
# u x r of a weight's gradient is positive: what is left out is missing from the sum in full.
GRADS = [("bf16", 64, 64, 3, 2, 12007), ("bf16", 128, 64, 3, 2, 12007), ("bf16", 48, 24, 3, 2, 12007),
         ("f32", 64, 64, 5, 2, 4001), ("f32", 16, 8, 2, 2, 20011), ("bf16", 64, 0, 19, 5, 1703)]


@pytest.mark.parametrize("size", GRADS)
@pytest.mark.parametrize("wanted", ["q", "k", "both"])
@pytest.mark.parametrize("by_head", [(False, False), (True, True), (True, False), (False, True)])
def test_weights_gradients_without_cancelling(size, wanted, by_head):
    dtype, D, R, H, Hk, T = size
    g = torch.Generator("cuda").manual_seed(D + R)
    B = 2
    xs = [rows(g, dtype, B, n, T, D) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(T, R, device="cuda") if R else (None, None)
    with torch.no_grad():
        dys = [y * (0.5 + i) for i, y in enumerate(da.qk_norm_rotary(*xs, cos, sin, norm=None))]
    w = [(1 + 0.3 * torch.randn(*((n, D) if per else (D,)), generator=g, device="cuda")) for n, per in zip((H, Hk), by_head)]
    asked = [i for i, name in enumerate("qk") if wanted in (name, "both")]
    for i in asked:
        w[i].requires_grad_()
    outs = da.qk_norm_rotary(*(x.requires_grad_() for x in xs), cos, sin, q_weight=w[0], k_weight=w[1], norm_eps=EPS)
    grads = torch.autograd.grad(outs, [w[i] for i in asked], dys)
    pos = torch.arange(T)[None].expand(B, T)
    for i, got in zip(asked, grads):
        n, parts, tail = (H, Hk)[i], [], []
        for x, dy in list(zip(xs, dys))[i::2]:
            args = (d64(w[i]), d64(cos), d64(sin))
            _, dw, size_ = ref.norm_rotate_backward(d64(x), *args, pos, False, "rms", EPS, d64(dy))
            parts.append((dw, size_))
            _, last, _ = ref.norm_rotate_backward(d64(x[:, :, -96:]), *args, pos[:, -96:], False, "rms", EPS, d64(dy[:, :, -96:]))
            tail.append(last)
        want, terms = (sum(p[j] for p in parts) for j in (0, 1))       # [heads, D]
        least = torch.stack([p[0] for p in parts]).amin(0)              # of a head of a tensor
        last = torch.stack(tail).amin(0)                                # of 192 tokens of one (96 a sequence)
        if not by_head[i]:
            want, terms, least, last = want.sum(0), terms.sum(0), least.amin(0), last.amin(0)
        # A term is off by (D/2 + 10) u of twice its size at most (the pair's other part may be the
        # larger: counted by max over channels).  The sums: a thread's over its tokens (3, or T B / 8
        # over the blocks of a head: 200 at most here), up to 5 exchanges, 8 warps, then up to 1,000
        # partial rows over 8 to 32 threads or more and those: fewer than 1,000 additions in a row.
        tol = ref.U * ((2 * D + 40) * terms.amax(-1, keepdim=True) + 1000 * terms)
        assert ((d64(got) - want).abs() <= tol).all(), "qk"[i]
        # and the bound is one that a missing part would break, in every channel
        assert (tol < least / 4).all() and (tol < last / 4).all()
