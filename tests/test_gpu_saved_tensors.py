"""GPU tests of the operators' gradients where hooks of saved tensors give them back in another
layout (save_on_cpu does): the same bits as without hooks, and an error for what was not saved."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod

pytestmark = pytest.mark.gpu
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


def reversed_order(t):
    """The first dimension innermost."""
    order = tuple(range(t.dim()))[::-1]
    return t.permute(order).contiguous().permute(order)


def swapped(t):
    """Dense, with the second and third dimensions swapped in memory."""
    return t.transpose(1, 2).contiguous().transpose(1, 2) if t.dim() == 4 else t.clone()


def odd_rows(t):
    """Rows of one element more than theirs, the rest of the store NaN."""
    if t.dim() == 0 or not t.is_floating_point():
        return t.clone()
    big = torch.full((*t.shape[:-1], t.shape[-1] + 1), float("nan"), dtype=t.dtype, device=t.device)
    big[..., :-1] = t
    return big[..., :-1]


def shifted(t):
    """Contiguous, but not from a 16-byte boundary."""
    big = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    big[1:] = t.reshape(-1)
    return big[1:].view(t.shape)


def unpacked(f):
    return lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach(), f)


HOOKS = {
    "cpu": lambda: torch.autograd.graph.save_on_cpu(),
    "pinned": lambda: torch.autograd.graph.save_on_cpu(pin_memory=True),
    "contiguous": unpacked(lambda t: t.clone(memory_format=torch.contiguous_format)),
    "reversed": unpacked(reversed_order),
    "swapped": unpacked(swapped),
    "odd": unpacked(odd_rows),
    "shifted": unpacked(shifted),
}


def projected(g, dtype, layout, B, T, widths):
    """Rows [B, heads, T, width] for each (heads, width): "token": [B, T, heads, width] seen so;
    "fused": slices of one projection [B, T, all of them]; "dense"."""
    if layout == "fused":
        total = sum(h * w for h, w in widths)
        store = torch.randn(B, T, total, generator=g).to(dtype).cuda()
        out, at = [], 0
        for h, w in widths:
            out.append(store[:, :, at:at + h * w].view(B, T, h, w).transpose(1, 2))
            at += h * w
        return out
    rows = [torch.randn(B, T, h, w, generator=g).to(dtype).cuda().transpose(1, 2) for h, w in widths]
    return rows if layout == "token" else [t.contiguous() for t in rows]


@pytest.mark.parametrize("hook", HOOKS)
@pytest.mark.parametrize("layout", ["token", "fused", "dense"])
@pytest.mark.parametrize("dtype,D,Dv,shared", [(BF, 64, 128, False), (BF, 64, 128, True), (BF, 128, 128, True), (F32, 32, 64, False),
                                               (BF, 128, 128, False), (F32, 20, 33, True)])
def test_cross_attention(hook, layout, dtype, D, Dv, shared):
    g = torch.Generator().manual_seed(D + Dv)
    B, H, Hk, Tq, Tk = 3, 4, 2, 70, 90
    q1, q2 = projected(g, dtype, layout, B, Tq, [(H, D), (H, D)])
    k1, k2, v = projected(g, dtype, layout, B, Tk, [(Hk, D), (Hk, D), (Hk, Dv)])
    leaves = [t.detach().requires_grad_() for t in ((q1, k1, q2, v) if shared else (q1, k1, q2, k2, v))]
    n = torch.tensor([90, 0, 33], dtype=torch.int32, device="cuda")
    do = torch.randn(B, H, Tq, Dv, generator=g).to(dtype).cuda()
    for lam in (torch.tensor(0.8, device="cuda"), torch.tensor(0.8, dtype=dtype, device="cuda")):
        lam.requires_grad_()

        def step():
            x = leaves[:3] + ([leaves[1]] if shared else [leaves[3]]) + leaves[-1:]
            return da.differential_cross_attention(*x, lam, kv_lengths=n)
        o = step()
        want = torch.autograd.grad(o, leaves + [lam], do)
        with HOOKS[hook]():
            o2 = step()
        got = torch.autograd.grad(o2, leaves + [lam], do)
        assert torch.equal(o, o2)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("change", [lambda t: t.cpu(), lambda t: t[..., :-1] if t.dim() else t.cpu(), lambda t: t.double()])
def test_cross_attention_refuses_what_was_not_saved(change):
    g = torch.Generator().manual_seed(1)
    q1, q2 = projected(g, BF, "token", 2, 20, [(4, 64), (4, 64)])
    k1, k2, v = projected(g, BF, "token", 2, 30, [(2, 64), (2, 64), (2, 128)])
    leaves = [t.detach().requires_grad_() for t in (q1, k1, q2, k2, v)]
    with unpacked(change)():
        o = da.differential_cross_attention(*leaves, 0.8)
    with pytest.raises(RuntimeError, match="hook of saved tensors"):
        torch.autograd.grad(o, leaves, torch.ones_like(o))


def spread(t):
    """Whole numbers as every other element of a larger store, the rest out of range."""
    if t.is_floating_point():
        return t.clone()
    big = torch.full((*t.shape[:-1], 2 * t.shape[-1]), 2 ** 30, dtype=t.dtype, device=t.device)
    big[..., ::2] = t
    return big[..., ::2]


DENSE_HOOKS = {**{k: HOOKS[k] for k in ("cpu", "pinned", "contiguous", "reversed", "swapped")}, "spread": unpacked(spread)}


@pytest.mark.parametrize("hook", DENSE_HOOKS)
@pytest.mark.parametrize("sections", [None, (8, 12, 12), (3, 18, 11)])
@pytest.mark.parametrize("batched", [False, True])
@pytest.mark.parametrize("dtype,whole", [(BF, torch.int64), (F32, torch.int32)])
def test_norm_and_rotation(hook, sections, batched, dtype, whole):
    """Positions as views: [axes, (B,) T] seen with the axes last, every third of a longer row."""
    g = torch.Generator().manual_seed(7)
    B, T, H, Hk, D = 2, 37, 4, 2, 64
    q1, k1, q2, k2 = (t.detach().requires_grad_() for t in projected(g, dtype, "token", B, T, [(H, D), (Hk, D), (H, D), (Hk, D)]))
    store = torch.randint(0, 90, (3, B, 3 * T), generator=g).to(whole).cuda()
    positions = (store if sections else store[:1])[:, :, ::3]
    positions = positions if batched else positions[:, 1]
    positions = positions.permute(*range(1, positions.dim()), 0) if sections else positions[0]
    cos, sin = da.rotary_tables(90, D, device="cuda", sections=sections)
    w = (1 + 0.2 * torch.randn(H, D, generator=g)).cuda().requires_grad_()
    leaves = [q1, k1, q2, k2, w]

    def step():
        return da.qk_norm_rotary(q1, k1, q2, k2, cos, sin, positions, q_weight=w, sections=sections)
    do = [torch.randn(t.shape, generator=g).to(dtype).cuda() for t in leaves[:4]]
    want = torch.autograd.grad(step(), leaves, do)
    with DENSE_HOOKS[hook]():
        y = step()
    for a, b in zip(torch.autograd.grad(y, leaves, do), want):
        assert torch.equal(a, b)


def test_norm_and_rotation_refuses_positions_that_were_not_saved():
    g = torch.Generator().manual_seed(8)
    q1, k1 = (t.detach().requires_grad_() for t in projected(g, BF, "token", 2, 9, [(4, 64), (2, 64)]))
    cos, sin = da.rotary_tables(20, 64, device="cuda")
    positions = torch.arange(9, device="cuda")
    for change in (lambda t: t if t.is_floating_point() else t.cpu(), lambda t: t if t.is_floating_point() else t[:5],
                   lambda t: t if t.is_floating_point() else t.int(), lambda t: t if t.shape != cos.shape else t[:3]):
        with unpacked(change)():
            y = da.qk_norm_rotary(q1, k1, None, None, cos, sin, positions)
        with pytest.raises(RuntimeError, match="hook of saved tensors"):
            torch.autograd.grad(y[:2], (q1, k1), (torch.ones_like(q1), torch.ones_like(k1)))


@pytest.mark.parametrize("change", [lambda t: t.cpu(), lambda t: t[:1], lambda t: t.double()])
@pytest.mark.parametrize("which", ["rows", "weight"])
def test_rows_and_weights_that_were_not_saved(change, which):
    g = torch.Generator().manual_seed(9)
    x, = (t.detach().requires_grad_() for t in projected(g, BF, "token", 2, 9, [(4, 64)]))
    w = torch.ones(4, 64, device="cuda", requires_grad=True)
    only = lambda t: change(t) if (t.dim() == 4) == (which == "rows") else t            # noqa: E731
    for f in (lambda: da.qk_norm_rotary(x, None, None, None, None, None, q_weight=w)[0],
              lambda: da.differential_head_norm(x, norm_weight=w)):
        with unpacked(only)():
            y = f()
        with pytest.raises(RuntimeError, match="hook of saved tensors"):
            torch.autograd.grad(y, (x, w), torch.ones_like(y))


@pytest.mark.parametrize("hook", ["cpu", "pinned", "contiguous", "reversed", "swapped"])
@pytest.mark.parametrize("layout", ["token", "fused", "dense"])
@pytest.mark.parametrize("dtype,norm", [(BF, "rms"), (BF, "group"), (F32, "group")])
def test_head_norm(hook, layout, dtype, norm):
    g = torch.Generator().manual_seed(10)
    x, _ = (t.detach().requires_grad_() for t in projected(g, dtype, layout, 3, 50, [(4, 128), (2, 64)]))
    w, b = ((1 + 0.2 * torch.randn(4, 128, generator=g)).cuda().requires_grad_() for _ in range(2))
    do = torch.randn(x.shape, generator=g).to(dtype).cuda()
    f = lambda: da.differential_head_norm(x, norm=norm, norm_weight=w, norm_bias=b, out_scale=0.2)      # noqa: E731
    want = torch.autograd.grad(f(), (x, w, b), do)
    with HOOKS[hook]():
        y = f()
    for a, c in zip(torch.autograd.grad(y, (x, w, b), do), want):
        assert torch.equal(a, c)


@pytest.mark.parametrize("dtype,D,Dv", [(BF, 64, 128), (BF, 128, 128), (F32, 32, 64)])
def test_recomputed_block(dtype, D, Dv):
    """Rotation, attention and head norm under activation checkpointing: the bits of the block itself."""
    from torch.utils.checkpoint import checkpoint
    g = torch.Generator().manual_seed(11)
    q1, q2 = projected(g, dtype, "fused", 2, 40, [(4, D), (4, D)])
    k, v = projected(g, dtype, "fused", 2, 70, [(2, D), (2, Dv)])
    leaves = [t.detach().requires_grad_() for t in (q1, k, q2, v)] + [torch.tensor(0.8, dtype=dtype, device="cuda").requires_grad_()]
    cos, sin = da.rotary_tables(90, D, device="cuda")
    n = torch.tensor([70, 31], dtype=torch.int32, device="cuda")

    def block(q1, k, q2, v, lam):
        q1, _, q2, _ = da.qk_norm_rotary(q1, None, q2, None, cos, sin)
        return da.differential_head_norm(da.differential_cross_attention(q1, k, q2, None, v, lam, kv_lengths=n), out_scale=0.2)
    do = torch.randn(2, 4, 40, Dv, generator=g).to(dtype).cuda()
    want = torch.autograd.grad(block(*leaves), leaves, do)
    got = torch.autograd.grad(checkpoint(block, *leaves, use_reentrant=False), leaves, do)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
