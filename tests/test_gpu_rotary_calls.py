"""GPU tests of calls of qk_norm_rotary and paged_cache_append that their signatures allow
beside the ordinary ones: what is refused, what is left out, what autograd keeps."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
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


def rows(g, B, H, T, D, dtype=torch.float32):
    return torch.randn(B, T, H, D, generator=g).to(dtype).cuda().transpose(1, 2)


def d64(t):
    return t.detach().cpu().double()


@pytest.mark.parametrize("D", [64, 48])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("side", ["q", "k"])
def test_a_weight_whose_rows_are_left_out(D, per_head, side):
    """Both weights trainable, rows of one kind alone: the other weight is not used, as in a
    formula that does not name it, and the used one's gradient is the formula's."""
    g = torch.Generator().manual_seed(D)
    B, T, H, Hk = 2, 7, 3, 2
    n = H if side == "q" else Hk
    xs = [rows(g, B, n, T, D) for _ in range(2)]
    used = (1 + 0.3 * torch.randn(*((n, D) if per_head else (D,)), generator=g)).cuda().requires_grad_()
    other = torch.ones(*((5, D) if per_head else (D,)), device="cuda", requires_grad=True)
    cos, sin = da.rotary_tables(T, D, device="cuda")
    args = (xs[0], None, xs[1], None) if side == "q" else (None, xs[0], None, xs[1])
    weights = dict(q_weight=used, k_weight=other) if side == "q" else dict(q_weight=other, k_weight=used)
    out = [y for y in da.qk_norm_rotary(*args, cos, sin, norm_eps=EPS, **weights) if y is not None]
    dys = [torch.randn(y.shape, generator=g).cuda() for y in out]
    got, none = torch.autograd.grad(out, [used, other], dys, retain_graph=True, allow_unused=True)
    assert none is None
    torch.autograd.backward(out, dys)
    assert other.grad is None and torch.equal(used.grad, got)
    pos = torch.arange(T)[None].expand(B, T)
    want = size = 0
    for x, dy in zip(xs, dys):
        _, dw, s = ref.norm_rotate_backward(d64(x), d64(used), d64(cos), d64(sin), pos, False, "rms", EPS, d64(dy))
        want, size = want + (dw if per_head else dw.sum(0)), size + (s if per_head else s.sum(0))
    # a term is off by (D/2 + 10) u of twice its size at most, a sum of N terms by N u
    terms = 2 * B * T * (1 if per_head else n)
    assert ((d64(got) - want).abs() <= ref.U * ((2 * D + 40) * size.amax(-1, keepdim=True) + terms * size)).all()
    # a weight that is not used asks for no graph
    alone = dict(q_weight=used.detach(), k_weight=other) if side == "q" else dict(q_weight=other, k_weight=used.detach())
    assert not any(y.requires_grad for y in da.qk_norm_rotary(*args, cos, sin, **alone) if y is not None)
    # and is looked at all the same
    bad = "k_weight" if side == "q" else "q_weight"
    for w in (torch.ones(D + 1, device="cuda"), torch.ones(2, D + 1, device="cuda"), torch.ones(D)):
        with pytest.raises(ValueError, match=bad):
            da.qk_norm_rotary(*args, cos, sin, **{bad: w})


def test_dual_tensors_are_refused():
    """Forward-mode differentiation: a result without a tangent would be a derivative of zero."""
    import torch.autograd.forward_ad as fwad
    g = torch.Generator().manual_seed(1)
    B, H, T, D, page = 2, 2, 3, 64, 16
    q, k = rows(g, B, H, T, D, torch.bfloat16), rows(g, B, H, T, D, torch.bfloat16)
    v = rows(g, B, H, T, 2 * D, torch.bfloat16)
    w = torch.ones(D, device="cuda")
    cos, sin = da.rotary_tables(page, D, device="cuda")
    kc, vc = (torch.zeros(B, H, page, n, dtype=torch.bfloat16, device="cuda") for n in (D, 2 * D))
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    nw = torch.ones(H, 2 * D, device="cuda")
    lam = torch.tensor(0.5, device="cuda")
    out = torch.empty(B, H, T, 2 * D, dtype=torch.bfloat16, device="cuda")
    calls = [
        (lambda q, k, c, s, qw, kw: da.qk_norm_rotary(q, k, q, None, c, s, q_weight=qw, k_weight=kw), [q, k, cos, sin, w, w]),
        (lambda k, v, kc, vc, c, s, kw: da.paged_cache_append(k, None, v, kc, None, vc, table, lens, None, c, s, norm="rms",
                                                              k_weight=kw), [k, v, kc, vc, cos, sin, w]),
        (lambda q, kc, vc, lam, nw, nb, out: da.differential_attention_paged(
            q, kc, q, None, vc, table, lens, lam, norm="rms", norm_weight=nw, norm_bias=nb, out=out),
         [q, kc, vc, lam, nw, nw, out]),
        (lambda q, kc, vc, lam: da.differential_attention_tree(
            q, kc, q, None, vc, table, lens, torch.ones(T, T, dtype=torch.bool, device="cuda"), lam), [q, kc, vc, lam]),
    ]
    for call, args in calls:
        call(*args)
        for i, a in enumerate(args):
            with fwad.dual_level():
                duals = [fwad.make_dual(a, torch.ones_like(a)) if j == i else x for j, x in enumerate(args)]
                for grad in (True, False):              # forward mode has a switch of its own
                    with torch.set_grad_enabled(grad), pytest.raises(ValueError, match="forward-mode"):
                        call(*duals)
        torch.cuda.synchronize()
    # a dual level with no dual tensor among the arguments, and one that is over
    with fwad.dual_level():
        want = da.qk_norm_rotary(q, None, None, None, cos, sin)[0]
        fwad.make_dual(q, torch.ones_like(q))
    assert torch.equal(da.qk_norm_rotary(q, None, None, None, cos, sin)[0], want)


@pytest.mark.parametrize("D,R", [(64, 64), (48, 24)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_changed_in_place_after_a_rotation(D, R, interleaved):
    """Without the norm the gradient does not depend on the rows: they are not kept, and may be
    changed; with it a change is an error."""
    g = torch.Generator().manual_seed(D)
    B, H, Hk, T = 2, 3, 2, 9
    xs = [rows(g, B, n, T, D, torch.bfloat16) for n in (H, Hk, H, Hk)]
    cos, sin = da.rotary_tables(T, R, device="cuda")
    pos = torch.arange(T)[None].expand(B, T)

    def call(norm):
        leaves = [x.clone().requires_grad_() for x in xs]
        inner = [x * 1 for x in leaves]                 # not leaves: these may change in place
        args = dict(norm=norm, norm_eps=EPS, interleaved=interleaved)
        saved = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t.dim()) or t, lambda t: t):
            da.qk_norm_rotary(*inner, cos, sin, **args)
        assert saved.count(4) == (4 if norm else 0)
        out = da.qk_norm_rotary(*inner, cos, sin, **args)
        with torch.no_grad():
            for x in inner:
                x.fill_(float("nan"))
        return leaves, out

    leaves, out = call(None)
    # one output is not used: a gradient that never comes is zero
    dys = [torch.randn(y.shape, generator=g).to(torch.bfloat16).cuda() for y in out[:3]]
    grads = torch.autograd.grad(out[:3], leaves, dys)
    assert torch.count_nonzero(grads[3]) == 0
    for dx, dy in zip(grads, dys):
        want, _, _ = ref.norm_rotate_backward(None, None, d64(cos), d64(sin), pos, interleaved, None, EPS, d64(dy))
        # three float32 roundings of |dy_a| + |dy_b| <= 2 max|dy|, and the result's
        bound = 3 * ref.U * 2 * d64(dy).abs().amax(-1, keepdim=True) + 2.0 ** -8 * want.abs()
        assert ((d64(dx) - want).abs() <= bound).all()
    leaves, out = call("rms")
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out, leaves, [torch.ones_like(y) for y in out])


def test_interleaved_that_is_no_truth_value():
    g = torch.Generator().manual_seed(1)
    k, v = rows(g, 1, 2, 3, 64), rows(g, 1, 2, 3, 128)
    kc, vc = (torch.zeros(2, 2, 16, n, device="cuda") for n in (64, 128))
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    cos, sin = da.rotary_tables(16, 64, device="cuda")
    several = torch.zeros(2)
    with pytest.raises(TypeError, match="interleaved"):
        da.qk_norm_rotary(k, None, None, None, cos, sin, interleaved=several)
    with pytest.raises(TypeError, match="interleaved"):
        da.paged_cache_append(k, None, v, kc, None, vc, table, lens, None, cos, sin, interleaved=several)
    assert torch.count_nonzero(kc) == 0
    a, b = (da.qk_norm_rotary(k, None, None, None, cos, sin, interleaved=i)[0] for i in (1, True))
    assert torch.equal(a, b)
