"""GPU tests of differential_cross_attention, forward and backward, against its formulas in
float64.  tests/block_reference.py derives each element's bound."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import block_reference as ref

pytestmark = pytest.mark.gpu
H_OF = {torch.bfloat16: 2.0 ** -8, torch.float32: ref.U}
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
    return t.detach().cpu().double()


def check(name, got, want, tol):
    got = d64(got)
    assert got.shape == want.shape, name
    worst = ((got - want).abs() - tol - 1e-30).max()
    assert not worst > 0 and not got.isnan().any(), f"{name}: {worst.item():.3g} beyond its bound"


def inputs(seed, dtype, B, H, Hk, Tq, Tk, D, Dv, shared, lens=None, layout="dense", poison=True):
    """q1, k1, q2, k2, v and kv_lengths; NaN and infinities behind each sequence's states."""
    g = torch.Generator().manual_seed(seed)

    def rows(heads, T, width):
        t = torch.randn(B, heads, T, width, generator=g).to(dtype).cuda()
        if layout == "token":                       # [B, T, heads, width] seen as [B, heads, T, width]
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "odd":                         # a row stride that no vector load takes
            big = torch.full((B, heads, T, width + 1), float("nan"), dtype=dtype, device="cuda")
            big[..., :width] = t
            t = big[..., :width]
        return t
    x = [rows(H, Tq, D), rows(Hk, Tk, D), rows(H, Tq, D), None, rows(Hk, Tk, Dv)]
    x[3] = x[1] if shared else rows(Hk, Tk, D)
    n = None
    if lens is not None:
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for t in {id(t): t for t in (x[1], x[3], x[4])}.values():
            for b, k in enumerate(lens):
                if poison and k < Tk:
                    t[b, :, k:] = float("nan")
                    t[b, :, k::2] = float("inf")
    return x, n


def reference(x, lam, lens, saved=True):
    clean = [torch.nan_to_num(d64(t), 0.0, 0.0, 0.0) for t in x]
    return ref.Cross(*clean, lam, lens or [x[1].shape[2]] * x[1].shape[0], H_OF[x[0].dtype], saved)


def train(x, n, lam, do):
    leaves = [x[0], x[1], x[2]] + ([] if x[3] is x[1] else [x[3]]) + [x[4]]
    for t in leaves:
        t.requires_grad_()
    lam_t = torch.tensor(lam, device="cuda", requires_grad=True)
    o = da.differential_cross_attention(*x, lam_t, kv_lengths=n)
    grads = torch.autograd.grad(o, leaves + [lam_t], do)
    names = ["q1", "k1", "q2"] + ([] if x[3] is x[1] else ["k2"]) + ["v", "lam"]
    for t in leaves:
        t.requires_grad_(False)
    return o.detach(), dict(zip(names, grads))


def compare(x, n, lens, lam, seed=0):
    g = torch.Generator().manual_seed(seed + 99)
    B, H, Tq, _ = x[0].shape
    do = torch.randn(B, H, Tq, x[4].shape[3], generator=g).to(x[0].dtype).cuda()
    lam = float(torch.tensor(lam, dtype=torch.float32))
    o, grads = train(x, n, lam, do)
    with torch.no_grad():
        served = da.differential_cross_attention(*x, lam, kv_lengths=n)
    want = reference(x, lam, lens)
    check("o", o, want.o, want.o_tol)
    check("served o", served, want.o, want.o_tol)
    back = want.backward(d64(do))
    if x[3] is x[1]:
        back["k1"] = back["k"]
    for name, got in grads.items():
        check("d" + name, got, *back[name])
    for b, k in enumerate(lens or []):              # states that are not there, and rows over none
        for name in ("k1", "k2", "v"):
            assert name not in grads or not grads[name][b, :, k:].any()
        if k == 0:
            assert not o[b].any() and not served[b].any() and not grads["q1"][b].any() and not grads["q2"][b].any()
    return o, served, grads


WIDE = [(BF, 64, 128), (BF, 128, 128), (F32, 32, 64), (F32, 64, 128), (F32, 128, 256), (BF, 32, 64), (BF, 48, 30),
        (F32, 10, 7), (BF, 128, 256), (F32, 1, 1), (BF, 64, 64)]


@pytest.mark.parametrize("dtype,D,Dv", WIDE)
@pytest.mark.parametrize("shared", [False, True])
def test_widths(dtype, D, Dv, shared):
    lens = [75, 0, 33]
    x, n = inputs(D + Dv, dtype, 3, 4, 2, 41, 75, D, Dv, shared, lens)
    compare(x, n, lens, 0.8)


@pytest.mark.parametrize("dtype,D,Dv,shared", [(BF, 64, 128, False), (BF, 64, 128, True), (BF, 128, 128, True), (F32, 32, 64, False)])
@pytest.mark.parametrize("Tq,Tk,lens", [
    (1, 1, [1, 1]), (1, 77, None), (3, 64, [64, 63]), (130, 5, [5, 1]), (128, 128, [128, 65]), (257, 65, [1, 64]),
    (7, 300, [300, 129]), (300, 513, [512, 0]), (64, 64, None), (129, 200, [0, 0])])
def test_lengths(dtype, D, Dv, shared, Tq, Tk, lens):
    x, n = inputs(Tq + Tk, dtype, 2, 4, 4, Tq, Tk, D, Dv, shared, lens)
    compare(x, n, lens, 0.3)


@pytest.mark.parametrize("D,shared", [(64, False), (64, True), (128, True)])
@pytest.mark.parametrize("H,Hk,Tq,Tk,lens", [(2, 1, 700, 130, [130, 0]), (1, 1, 1100, 20, [20, 7]), (2, 2, 600, 300, [1, 300])])
def test_query_rows_in_splits(D, shared, H, Hk, Tq, Tk, lens):
    """Few tiles of states: dK and dV come from several blocks' partial sums."""
    x, n = inputs(Tq, BF, 2, H, Hk, Tq, Tk, D, 128, shared, lens)
    o, _, first = compare(x, n, lens, 0.8)
    do = torch.randn(o.shape, device="cuda").to(BF)
    first, again = train(x, n, 0.8, do)[1], train(x, n, 0.8, do)[1]
    assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (6, 3), (16, 2)])
@pytest.mark.parametrize("dtype,D,Dv,shared", [(BF, 64, 128, False), (BF, 128, 128, True), (F32, 64, 128, False)])
@pytest.mark.parametrize("Tq", [1, 70])
def test_grouped_heads(H, Hk, dtype, D, Dv, shared, Tq):
    lens = [130, 200]
    x, n = inputs(H, dtype, 2, H, Hk, Tq, 200, D, Dv, shared, lens)
    compare(x, n, lens, 0.8)


@pytest.mark.parametrize("H,Hk", [(16, 4), (18, 3), (32, 1), (10, 5), (16, 16)])
@pytest.mark.parametrize("D,shared", [(64, False), (128, True)])
@pytest.mark.parametrize("Tq", [1, 8, 9, 33, 64, 65])
def test_short_rows_of_many_heads(H, Hk, D, shared, Tq):
    """More heads than SMs: items take several heads of a group."""
    B = 160 // H + 2
    lens = [70, 0, 64, 3] + [70] * (B - 4)
    x, n = inputs(Tq, BF, B, H, Hk, Tq, 70, D, 128, shared, lens)
    compare(x, n, lens, 0.8)
    w = 1 + torch.arange(H * 128, device="cuda").reshape(H, 128) / 1000
    with torch.no_grad():                           # a weight a head, and rows of their own strides
        out = torch.full((B, Tq, H, 128), 7.0, dtype=BF, device="cuda").transpose(1, 2)
        got = da.differential_cross_attention(*x, 0.8, kv_lengths=n, norm="rms", norm_weight=w, out_scale=0.5, out=out)
        one = torch.cat([da.differential_cross_attention(*[t[b:b + 1] for t in x], 0.8, kv_lengths=n[b:b + 1], norm="rms",
                                                         norm_weight=w, out_scale=0.5) for b in range(B)])
    # one sequence may go another way: each is within its bound, which a norm of O spreads over the row
    o = reference(x, float(torch.tensor(0.8)), lens)
    rs = (o.o.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt()
    tol = o.o_tol - o.h * o.o.abs()
    tol = 1.5 * rs * (tol + o.o.abs() * rs * rs * (o.o.abs() * tol).mean(-1, keepdim=True)) + 64 * ref.U
    check("normed", got, d64(one), 2 * 0.5 * d64(w)[:, None] * tol + 4 * o.h * d64(one).abs())


@pytest.mark.parametrize("layout", ["token", "odd"])
@pytest.mark.parametrize("dtype,D,Dv,shared", [(BF, 64, 128, False), (BF, 128, 128, True), (F32, 64, 128, False)])
def test_layouts(layout, dtype, D, Dv, shared):
    lens = [90, 17]
    x, n = inputs(3, dtype, 2, 4, 2, 40, 90, D, Dv, shared, lens, layout)
    compare(x, n, lens, 0.8)


@pytest.mark.parametrize("lam", [0.0, 1.0, -0.35, 1.7])
def test_coefficients(lam):
    lens = [90, 64]
    x, n = inputs(4, BF, 2, 4, 2, 40, 90, 64, 128, False, lens)
    compare(x, n, lens, lam)


@pytest.mark.parametrize("dtype,D,Dv", [(BF, 64, 128), (BF, 128, 128), (F32, 64, 128)])
@pytest.mark.parametrize("Tq", [1, 20, 200])
def test_alike_branches_cancel(dtype, D, Dv, Tq):
    x, n = inputs(5, dtype, 2, 4, 2, Tq, 150, D, Dv, True, [150, 31])
    x[2] = x[0]
    with torch.no_grad():
        assert not da.differential_cross_attention(*x, 1.0, kv_lengths=n).any()
    o, _ = train([x[0], x[1], x[0].clone(), x[1], x[4]], n, 1.0, torch.ones(2, 4, Tq, Dv, dtype=dtype, device="cuda"))
    assert not o.any()


@pytest.mark.parametrize("dtype,D,Dv", [(BF, 64, 128), (F32, 64, 128), (BF, 128, 128)])
@pytest.mark.parametrize("norm", ["rms", "group", None])
@pytest.mark.parametrize("Tq", [1, 33, 260])
def test_epilogue(dtype, D, Dv, norm, Tq):
    """The fused norm, weight, bias and scale, from the reference's O: its bound goes through
    the norm, whose own roundings are K = 32 U (as in the head norm's tests)."""
    lens = [100, 0, 64]
    x, n = inputs(6, dtype, 3, 4, 2, Tq, 100, D, Dv, True, lens)
    g = torch.Generator().manual_seed(7)
    w, b = (1 + 0.2 * torch.randn(4, Dv, generator=g)), 0.2 * torch.randn(4, Dv, generator=g)
    eps = 1e-3
    kw = {} if norm is None else dict(norm=norm, norm_eps=eps, norm_weight=w.cuda(), norm_bias=b.cuda())
    if norm is None:                                        # a scale alone
        w, b = torch.ones(4, Dv), torch.zeros(4, Dv)
    with torch.no_grad():
        y = da.differential_cross_attention(*x, 0.8, kv_lengths=n, out_scale=0.2, **kw)
    r = reference(x, float(torch.tensor(0.8)), lens)
    w, b = w.double()[:, None], b.double()[:, None]
    tol = r.o_tol - r.h * r.o.abs()                         # O is not rounded on the way
    o = r.o
    if norm is not None:
        if norm == "group":
            tol = tol + tol.mean(-1, keepdim=True)
            o = o - o.mean(-1, keepdim=True)
        rs = (o.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
        # h = o rs: its own error, and rs's through the mean square: d rs = rs^3 mean(o d o)
        hat = o * rs
        tol = rs * tol + hat.abs() * rs * rs * (o.abs() * tol).mean(-1, keepdim=True) + 32 * ref.U * (hat.abs() + r.o.abs().mean(-1, keepdim=True) * rs)
        # second order: the bound holds where a row's error is small beside its size
        tol = 1.5 * tol
        o = hat
    want = 0.2 * (o * w + b)
    check("y", y, want, 0.2 * (w.abs() * tol + 4 * ref.U * (b.abs() + (o * w).abs())) + r.h * want.abs())


@pytest.mark.parametrize("D,shared", [(64, False), (64, True), (128, True)])
@pytest.mark.parametrize("Tq,Tk", [(1, 300), (1, 4000), (9, 4000), (40, 300), (200, 300), (200, 64)])
@pytest.mark.parametrize("kind", ["alike", "late keys"])
def test_weights_in_two_parts(D, shared, Tq, Tk, kind):
    """On every route O is off by its own rounding and little else: each weight by 2^-16 (two bf16
    parts, half a step 2^-8 each), with branches that cancel, and with rows that attend to the
    keys 16 to 63 of each 64."""
    lens = [Tk, Tk // 4]
    x, n = inputs(23, BF, 2, 4, 2, Tq, Tk, D, 128, shared, lens)
    g = torch.Generator().manual_seed(24)
    if kind == "alike":
        x[0] = (2 * x[0]).contiguous()
        x[2] = x[0] + (0.2 * torch.randn(x[0].shape, generator=g)).to(BF).cuda()
        if not shared:
            x[3] = x[1] + (0.2 * torch.randn(x[1].shape, generator=g)).to(BF).cuda()
    else:                                           # a direction that queries share and late keys have
        u = torch.randn(D, generator=g).cuda()
        x[0], x[2] = (x[0] + u).to(BF), (x[2] + u).to(BF)
        late = (torch.arange(Tk, device="cuda") % 64 >= 16)[:, None] * (6 * D ** 0.5 / u.square().sum() * u)
        x[1] = (x[1] + late).to(BF)
        x[3] = x[1] if shared else (x[3] + late).to(BF)
    lam = float(torch.tensor(0.8))
    with torch.no_grad():
        got = da.differential_cross_attention(*x, lam, kv_lengths=n)
    clean = [torch.nan_to_num(d64(t), 0.0, 0.0, 0.0) for t in x]
    want = ref.Cross(*clean, lam, lens, 2.0 ** -16)
    check("o", got, want.o, want.o_tol + 2.0 ** -8 * want.o.abs())
    o, _ = train(x, n, lam, torch.ones(2, 4, Tq, 128, dtype=BF, device="cuda"))
    check("training o", o, want.o, want.o_tol + 2.0 ** -8 * want.o.abs())


@pytest.mark.parametrize("D,shared", [(64, False), (64, True), (128, True), (128, False)])
@pytest.mark.parametrize("Tk", [65, 130, 300, 1500])
@pytest.mark.parametrize("kind", ["offsets", "peaks", "alike"])
def test_query_gradients_where_rows_share_an_error(D, shared, Tk, kind):
    """dQ where keys and values have offsets, where one state takes nearly all of a row, and where
    the branches are alike, against what roundings of dS allow if each is its own.

    dS_j and dQ are rounded by 2^-8 at most each, of either sign, so that a row's error is a
    sum of independent terms e_j K_j with |e_j| <= 2^-8 |dS_j|: its squared norm is on average at
    most sum_j (2^-8 |dS_j| |K_j|)^2, and (2^-8 |dQ|)^2 for the result's.  (Uniform errors have a third of
    these squares, so a tensor of 400 rows stays below the sum, and a row below three times its root.)
    What a row's dS share, the error of Dd, is the bound of a forward that rounds by 2^-16."""
    lens = [Tk, Tk - 40]
    H, Tq = 2, 100
    x, n = inputs(25, BF, 2, H, 1, Tq, Tk, D, 128, shared, lens)
    g = torch.Generator().manual_seed(26)
    normal = lambda *shape: torch.randn(*shape, generator=g).cuda()                 # noqa: E731
    if kind == "offsets":
        x[1] = (x[1] + 2 * normal(D)).to(BF)
        x[3] = x[1] if shared else (x[3] + 2 * normal(D)).to(BF)
        x[4] = (x[4] + 2 * normal(128)).to(BF)
    else:
        x[0], x[2] = 4 * x[0], 4 * x[2]
        if kind == "alike":
            x[2] = (x[0] + 0.2 * normal(2, H, Tq, D)).to(BF)
            x[3] = x[1] if shared else (x[1] + 0.2 * normal(2, 1, Tk, D)).to(BF)
    lam = float(torch.tensor(0.8))
    do = torch.randn(2, H, Tq, 128, generator=g).to(BF).cuda()
    _, grads = train(x, n, lam, do)
    clean = [torch.nan_to_num(d64(t), 0.0, 0.0, 0.0) for t in x]
    want = ref.Cross(*clean, lam, lens, 2.0 ** -16)
    shares = want.backward(d64(do))
    for name, j in (("q1", 0), ("q2", 1)):
        w, share = shares[name]
        own = (2.0 ** -8 * w).square().sum(-1)
        for (b, i), (A, _, _, _) in want.heads.items():
            K = clean[1 + 2 * j][b, 0, :lens[b]]
            dP = d64(do)[b, i] @ clean[4][b, 0, :lens[b]].T
            dS = (1.0, lam)[j] * A[j] * (dP - (A[j] * dP).sum(-1, keepdim=True)) * D ** -0.5
            own[b, i] += (2.0 ** -8 * dS).square() @ K.square().sum(-1)
        err = (d64(grads[name]) - w)
        excess = (err.abs() - share).clamp(min=0).square().sum(-1)
        assert excess.sum() <= own.sum(), (name, excess.sum().item() / own.sum().item())
        assert (excess <= 9 * own + 1e-30).all(), (name, (excess / own).max().item())


def test_training_without_rests():
    """The C ABI's calls without the rests of the forward's roundings: a row's Dd from O and A_2 V as
    they were rounded."""
    import ctypes
    from differential_attention_fwd_gb300 import _lib
    lib = _lib.load()
    lens = [300, 140]
    for D, shared in ((64, False), (128, True)):
        x, n = inputs(27, BF, 2, 4, 2, 70, 300, D, 128, shared, lens)
        do = torch.randn(2, 4, 70, 128, device="cuda").to(BF)
        d = _lib.DiffattnCrossDesc()
        d.B, d.H, d.Tq, d.Tk, d.D, d.Dv, d.dtype, d.kv_group, d.lambda_dtype = 2, 4, 70, 300, D, 128, _lib.DIFFATTN_BF16, 2, _lib.DIFFATTN_F32
        o, o2 = torch.empty_like(do), torch.empty_like(do)
        lse = torch.empty(2, 4, 70, 2, device="cuda")
        for f, t in zip(("q1", "k1", "q2", "k2", "v", "o", "dout"), x + [o, do]):
            getattr(d, f + "_stride")[:] = t.stride()[:3]
        grads = [torch.empty_like(t) for t in x]
        if shared:
            grads[3] = None
        dlam = torch.empty((), device="cuda")
        p = lambda t: None if t is None else t.data_ptr()                           # noqa: E731
        ws = torch.empty(max(lib.diffattn_cross_workspace_bytes(ctypes.byref(d)), lib.diffattn_cross_bwd_workspace_bytes(ctypes.byref(d))),
                         dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.diffattn_cross_fwd(ctypes.byref(d), *map(p, x), p(n), 0.8, None, None, p(o), p(o2), p(lse), p(ws), ws.numel(), stream) == 0
        assert lib.diffattn_cross_bwd(ctypes.byref(d), *map(p, x), p(n), 0.8, None, p(o), p(o2), p(lse), p(do), *map(p, grads), p(dlam),
                                      p(ws), ws.numel(), stream) == 0
        want = reference(x, float(torch.tensor(0.8)), lens)
        back = want.backward(d64(do))
        if shared:
            back["k1"] = back["k"]
        check("o", o, want.o, want.o_tol)
        for name, t in zip(("q1", "k1", "q2", "k2", "v", "lam"), grads + [dlam]):
            if t is not None:
                check("d" + name, t, *back[name])


@pytest.mark.parametrize("norm", ["rms", "group"])
@pytest.mark.parametrize("D,shared", [(64, False), (128, True)])
@pytest.mark.parametrize("H,Hk,Tq", [(16, 16, 130), (16, 4, 20)])
def test_norm_between_sequences_without_states(norm, D, shared, H, Hk, Tq):
    """Several items an SM, with sequences of no state before and after each that has some: the rows
    have the bits of a call over the latter alone."""
    B = 96
    lens = [64 if b % 3 == 1 else 0 for b in range(B)]
    x, n = inputs(22, BF, B, H, Hk, Tq, 70, D, 128, shared, lens)
    some = [b for b in range(B) if lens[b]]
    y = [t[some].contiguous() for t in x]
    if shared:
        y[3] = y[1]
    w, b = 1 + torch.arange(H * 128, device="cuda").reshape(H, 128) / 1000, torch.ones(H, 128, device="cuda")
    kw = dict(norm=norm, norm_weight=w, norm_bias=b, out_scale=0.5)
    with torch.no_grad():
        want = da.differential_cross_attention(*y, 0.8, kv_lengths=n[some].contiguous(), **kw)
        for _ in range(20):
            got = da.differential_cross_attention(*x, 0.8, kv_lengths=n, **kw)
            assert torch.equal(got[some], want)
            assert (got[[b for b in range(B) if not lens[b]]] == 0.5).all()


def test_one_answer_for_full_lengths_and_none():
    for dtype, D, Dv in ((BF, 64, 128), (F32, 64, 128)):
        for Tq in (1, 40):
            x, _ = inputs(8, dtype, 2, 4, 2, Tq, 90, D, Dv, False)
            full = torch.full((2,), 90, dtype=torch.int32, device="cuda")
            with torch.no_grad():
                assert torch.equal(da.differential_cross_attention(*x, 0.8), da.differential_cross_attention(*x, 0.8, full))
                lens = torch.tensor([90, 0, 0, 90], dtype=torch.int32, device="cuda")[::3]      # not contiguous
                assert torch.equal(da.differential_cross_attention(*x, 0.8), da.differential_cross_attention(*x, 0.8, lens))


@pytest.mark.parametrize("dtype,D,Dv", [(BF, 64, 128), (F32, 64, 128), (BF, 128, 128)])
@pytest.mark.parametrize("Tq", [1, 40, 200])
def test_lengths_out_of_range(dtype, D, Dv, Tq):
    """A bad length: that sequence alone is NaN, and it is reported."""
    x, _ = inputs(9, dtype, 4, 4, 2, Tq, 90, D, Dv, True)
    good, bad = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([50, 90, 7, 90], [50, 91, 7, -1]))
    do = torch.randn(4, 4, Tq, Dv, device="cuda").to(dtype)
    want, wg = train(x, good, 0.8, do)
    with torch.no_grad():
        served = da.differential_cross_attention(*x, 0.8, kv_lengths=good)
    assert da.get_device_error() == 0
    got, gg = train(x, bad, 0.8, do)
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    with torch.no_grad():
        other = da.differential_cross_attention(*x, 0.8, kv_lengths=bad)
    assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX
    for a, b in [(got, want), (other, served)] + [(gg[k], wg[k]) for k in ("q1", "k1", "q2", "v")]:
        assert torch.equal(a[0::2], b[0::2]) and a[1::2].isnan().all()


def test_out_and_strided_results():
    x, n = inputs(10, BF, 2, 4, 2, 30, 90, 64, 128, False, [90, 0])
    with torch.no_grad():
        want = da.differential_cross_attention(*x, 0.8, kv_lengths=n)
        out = torch.full((2, 30, 4, 128), 7.0, dtype=BF, device="cuda").transpose(1, 2)
        assert da.differential_cross_attention(*x, 0.8, kv_lengths=n, out=out) is out and torch.equal(out, want)
        big = torch.full((2, 4, 30, 131), 7.0, dtype=BF, device="cuda")
        da.differential_cross_attention(*x, 0.8, kv_lengths=n, out=big[..., 1:129])
        assert (big[..., 0] == 7).all() and (big[..., 129:] == 7).all()
        check("odd out", big[..., 1:129], *(lambda r: (r.o, r.o_tol))(reference(x, float(torch.tensor(0.8)), [90, 0])))
        for Tq in (1, 5, 200):                  # every path of the same call
            y, m = inputs(11, BF, 2, 4, 2, Tq, 90, 64, 128, False, [90, 3])
            want = da.differential_cross_attention(*y, 0.8, kv_lengths=m)
            out = torch.full((2, Tq, 4, 128), 7.0, dtype=BF, device="cuda").transpose(1, 2)
            da.differential_cross_attention(*y, 0.8, kv_lengths=m, out=out)
            assert torch.equal(out, want)


def test_some_gradients_alone():
    """Frozen queries, a frozen encoder, a trained coefficient: what asks for a gradient gets the
    same one."""
    x, n = inputs(12, BF, 2, 4, 2, 70, 90, 64, 128, False, [90, 20])
    do = torch.randn(2, 4, 70, 128, device="cuda").to(BF)
    _, want = train(x, n, 0.8, do)
    names = ["q1", "k1", "q2", "k2", "v"]
    for which in (["q1"], ["q2", "lam"], ["k2"], ["v"], ["lam"], ["k1", "v"]):
        ts = [t.detach().requires_grad_(name in which) for name, t in zip(names, x)]
        lam = torch.tensor(0.8, device="cuda", requires_grad="lam" in which)
        o = da.differential_cross_attention(*ts, lam, kv_lengths=n)
        every = dict(zip(names + ["lam"], ts + [lam]))
        got = torch.autograd.grad(o, [every[w] for w in which], do)
        for w, g in zip(which, got):
            assert torch.equal(g, want[w]), w


@pytest.mark.parametrize("dtype,D,Dv", [(BF, 128, 128), (BF, 64, 128), (F32, 64, 128)])
@pytest.mark.parametrize("Tq", [20, 700])
def test_queries_alone_over_one_key_tensor(dtype, D, Dv, Tq):
    x, n = inputs(19, dtype, 2, 4, 2, Tq, 90, D, Dv, True, [90, 20])
    do = torch.randn(2, 4, Tq, Dv, device="cuda").to(dtype)
    _, want = train(x, n, 0.8, do)
    q1, q2 = x[0].clone().requires_grad_(), x[2].clone().requires_grad_()
    got = torch.autograd.grad(da.differential_cross_attention(q1, x[1], q2, x[1], x[4], 0.8, kv_lengths=n), (q1, q2), do)
    assert torch.equal(got[0], want["q1"]) and torch.equal(got[1], want["q2"])


@pytest.mark.parametrize("dtype,D,Dv,shared", [(BF, 64, 128, False), (BF, 128, 128, True), (F32, 32, 64, False)])
@pytest.mark.parametrize("H,Hk,Tq", [(4, 4, 1), (4, 2, 2), (4, 2, 3), (4, 4, 70)])
def test_states_that_all_sequences_read(dtype, D, Dv, shared, H, Hk, Tq):
    """One encoder's states expanded over the batch, and a gradient expanded over the heads: the
    answers of copies, and the states' gradients summed by autograd."""
    x, n = inputs(20, dtype, 3, H, Hk, Tq, 90, D, Dv, shared)
    n = torch.tensor([90, 0, 41], dtype=torch.int32, device="cuda")
    one = [t[:1].clone().requires_grad_() for t in (x[1], x[3], x[4])]
    k1 = one[0].expand(3, -1, -1, -1)
    k2 = k1 if shared else one[1].expand(3, -1, -1, -1)
    y = [x[0], k1, x[2], k2, one[2].expand(3, -1, -1, -1)]
    dense = [t.detach().contiguous() for t in y]
    dense[3] = dense[1] if shared else dense[3]
    do = torch.randn(3, 1, Tq, Dv, device="cuda").to(dtype).expand(-1, H, -1, -1)
    o = da.differential_cross_attention(*y, 0.8, kv_lengths=n)
    lens = n.tolist()
    lam = float(torch.tensor(0.8))
    want = reference(dense, lam, lens)
    check("o", o, want.o, want.o_tol)
    with torch.no_grad():
        check("served o", da.differential_cross_attention(*y, 0.8, kv_lengths=n), want.o, want.o_tol)
    got = torch.autograd.grad(o, one if not shared else [one[0], one[2]], do)
    back = want.backward(d64(do))
    names = ["k", "v"] if shared else ["k1", "k2", "v"]
    for name, g in zip(names, got):
        # the sum over the batch: each sequence's gradient was rounded, and so is the sum
        w, tol = back[name]
        check("d" + name, g, w.sum(0, keepdim=True), tol.sum(0, keepdim=True) + H_OF[dtype] * (w.sum(0, keepdim=True).abs() + tol.sum(0, keepdim=True)))


def test_coefficient_kinds():
    x, n = inputs(13, BF, 2, 4, 2, 20, 90, 64, 128, False, [90, 20])
    do = torch.randn(2, 4, 20, 128, device="cuda").to(BF)
    _, want = train(x, n, 0.75, do)
    with torch.no_grad():
        o = da.differential_cross_attention(*x, 0.75, kv_lengths=n)
        for lam in (torch.tensor(0.75), torch.tensor([[0.75]], dtype=torch.float64, device="cuda"), torch.tensor(0.75, device="cuda").bfloat16()):
            assert torch.equal(o, da.differential_cross_attention(*x, lam, kv_lengths=n))
    for lam in (torch.tensor(0.75), torch.tensor([0.75], dtype=torch.float64, device="cuda"), torch.tensor(0.75, device="cuda").bfloat16()):
        lam.requires_grad_()
        g, = torch.autograd.grad(da.differential_cross_attention(*x, lam, kv_lengths=n), lam, do)
        assert g.shape == lam.shape and g.dtype == lam.dtype and g.device == lam.device
        assert torch.equal(g.reshape(()).cpu(), want["lam"].cpu().to(lam.dtype))


def test_same_bits_on_other_streams_and_in_graphs():
    """Each time the same bits; calls on two streams at once; a captured training step replayed on
    new inputs and new lengths; two graphs that run at the same time."""
    x, n = inputs(14, BF, 3, 4, 2, 150, 300, 64, 128, False, [300, 120, 0], poison=False)
    do = torch.randn(3, 4, 150, 128, device="cuda").to(BF)
    o, want = train(x, n, 0.8, do)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(train(x, n, 0.8, do))
    torch.cuda.synchronize()
    for o2, g in got:
        assert torch.equal(o, o2) and all(torch.equal(want[k], g[k]) for k in want)
    leaves = [t.requires_grad_() for t in x]
    lam = torch.tensor(0.8, device="cuda")
    graphs, held = [], []
    with torch.cuda.stream(streams[0]):
        torch.autograd.grad(da.differential_cross_attention(*x, lam, kv_lengths=n), leaves, do)
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = da.differential_cross_attention(*x, lam, kv_lengths=n)
            gs = torch.autograd.grad(y, leaves, do)
            with torch.no_grad():
                served = da.differential_cross_attention(*[t[:, :, :1] if i in (0, 2) else t for i, t in enumerate(x)], lam, kv_lengths=n)
        graphs.append(graph)
        held.append((y, *gs, served))
    with torch.no_grad():
        for t in x:
            t.copy_(torch.randn_like(t))
    n.copy_(torch.tensor([0, 299, 64], dtype=torch.int32))
    torch.cuda.synchronize()
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    o3, g3 = train([t.detach() for t in x], n, 0.8, do)
    with torch.no_grad():
        served = da.differential_cross_attention(*[t[:, :, :1] if i in (0, 2) else t for i, t in enumerate(x)], lam, kv_lengths=n)
    for h in held:
        for a, b in zip(h, (o3, g3["q1"], g3["k1"], g3["q2"], g3["k2"], g3["v"], served)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,H,Hk,Tq,Tk,D", [(4, 16, 16, 700, 3000, 64), (3, 16, 8, 700, 3000, 128), (24, 16, 4, 20, 900, 64)])
def test_long_calls_in_graphs_and_at_once(B, H, Hk, Tq, Tk, D):
    """Items claimed from a counter, and several heads an item: two replayed graphs at once and two
    streams at once, on new lengths, have the bits of a call alone."""
    x, _ = inputs(21, BF, B, H, Hk, Tq, Tk, D, 128, D == 128)
    n = torch.full((B,), Tk, dtype=torch.int32, device="cuda")
    x = [t.requires_grad_() for t in x]
    leaves = x[:3] + ([] if D == 128 else [x[3]]) + [x[4]]
    do = torch.randn(B, H, Tq, 128, device="cuda").to(BF)
    lam = torch.tensor(0.8, device="cuda")

    def step():
        o = da.differential_cross_attention(*x, lam, kv_lengths=n)
        with torch.no_grad():
            served = da.differential_cross_attention(*x, lam, kv_lengths=n, norm="rms")
        return o, served, *torch.autograd.grad(o, leaves, do)
    streams = [torch.cuda.Stream() for _ in range(2)]
    with torch.cuda.stream(streams[0]):
        step()
    torch.cuda.synchronize()
    graphs, held = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append([t.detach() for t in step()])
        graphs.append(graph)
    n.copy_(torch.arange(B, dtype=torch.int32) * (Tk // B))         # the first without a state
    want = [t.detach() for t in step()]
    torch.cuda.synchronize()
    for _ in range(3):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for h in held:
        assert all(torch.equal(a, b) for a, b in zip(h, want))
    got = []
    for stream in streams:
        with torch.cuda.stream(stream):
            got.append(step())
    torch.cuda.synchronize()
    for h in got:
        assert all(torch.equal(a, b) for a, b in zip(h, want))
    assert not want[0][0].any() and want[0][-1].isfinite().all()


def test_non_finite_states_that_are_seen_stay_in_their_sequence():
    x, n = inputs(15, BF, 2, 4, 2, 40, 90, 64, 128, False, [90, 50], poison=False)
    with torch.no_grad():
        want = da.differential_cross_attention(*x, 0.8, kv_lengths=n)
        x[4][0, 0, 3, 5] = float("nan")
        x[1][0, 1, 4] = float("nan")
        got = da.differential_cross_attention(*x, 0.8, kv_lengths=n)
    assert torch.equal(got[1], want[1])
    assert got[0, :2, :, 5].isnan().all() and got[0, 2:].isnan().all()


def test_offsets_past_32_bits():
    """States of a batch more than 2^31 elements apart."""
    Tk, D, Dv = 70, 64, 128
    store = torch.zeros(2 ** 31 + 4096 + Tk * Dv, dtype=BF, device="cuda")
    x, _ = inputs(16, BF, 2, 2, 2, 40, Tk, D, Dv, True)
    far = 2 ** 31 + 4096
    for i, width in ((1, D), (4, Dv)):
        view = store.as_strided((2, 1, Tk, width), (far, Tk * width, width, 1), 0 if i == 1 else 0)
        view.copy_(x[i][:, :1])
        y = list(x)
        y[1] = y[3] = x[1][:, :1]
        y[4] = x[4][:, :1]
        with torch.no_grad():
            want = [da.differential_cross_attention(*[t[:, :, :q] if k in (0, 2) else t for k, t in enumerate(y)], 0.8) for q in (1, 40)]
            if i == 1:
                y[1] = y[3] = view
            else:
                y[4] = view
            got = [da.differential_cross_attention(*[t[:, :, :q] if k in (0, 2) else t for k, t in enumerate(y)], 0.8) for q in (1, 40)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_refusals():
    x, n = inputs(17, F32, 1, 2, 2, 5, 9, 32, 64, False)
    f = da.differential_cross_attention
    q = x[0].clone().requires_grad_()
    w = torch.ones(2, 64, device="cuda", requires_grad=True)
    for kw in (dict(norm="rms"), dict(out_scale=0.5), dict(out=torch.empty(1, 2, 5, 64, device="cuda"))):
        with pytest.raises(ValueError, match="bare operation"):
            f(q, *x[1:], 0.5, **kw)
    with pytest.raises(ValueError, match="bare operation"):
        f(*x, 0.5, norm="rms", norm_weight=w)
    o = f(q, *x[1:], 0.5)
    torch.autograd.grad(o, q, torch.ones_like(o))
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(o, q, torch.ones_like(o))
    o = f(q, *x[1:], 0.5)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(o, q, torch.ones_like(o), create_graph=True)
    o = f(q, *x[1:], 0.5)
    with torch.no_grad():
        o.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(o, q, torch.ones_like(o))
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ValueError, match="forward-mode"):
            f(torch.autograd.forward_ad.make_dual(x[0], x[0]), *x[1:], 0.5)


def test_refusals():
    x, _ = inputs(18, BF, 2, 4, 2, 5, 9, 64, 128, False)
    f = da.differential_cross_attention
    q1, k1, q2, k2, v = x
    lens = torch.tensor([9, 9], dtype=torch.int32, device="cuda")
    for bad in ((q1[0], k1, q2, k2, v), (q1, k1, q2[:, :2], k2, v), (q1, k1[:, :, :8], q2, k2, v), (q1, k1, q2, k2, v[:1]),
                (q1[:, :3], k1, q2[:, :3], k2, v), (q1.float(), k1, q2, k2, v), (q1.half(), k1.half(), q2.half(), k2.half(), v.half()),
                (q1, k1.cpu(), q2, k2, v), (q1[:, :, :0], k1, q2[:, :, :0], k2, v), (q1, k1[:, :, :0], q2, k2[:, :, :0], v[:, :, :0])):
        with pytest.raises(ValueError):
            f(*bad, 0.5)
    for kw in (dict(kv_lengths=lens.long()), dict(kv_lengths=lens[:1]), dict(kv_lengths=lens.cpu()), dict(norm="layer"),
               dict(out=torch.empty(2, 4, 5, 64, dtype=BF, device="cuda")), dict(norm="rms", norm_weight=torch.ones(3, 128, device="cuda")),
               dict(norm_weight=torch.ones(4, 128, device="cuda")), dict(norm="none", norm_bias=torch.ones(4, 128, device="cuda"))):
        with pytest.raises(ValueError):
            f(*x, 0.5, **kw)
    with pytest.raises(TypeError):
        f(*x, "0.5")
    with pytest.raises(TypeError):
        f(q1, None, q2, k2, v, 0.5)
    with pytest.raises(ValueError):
        f(*x, torch.ones(2))
    with pytest.raises(da.DiffattnError):
        f(*x, float("nan"))
    with pytest.raises(da.DiffattnError):
        f(*x, 0.5, out=torch.empty(1, 4, 5, 128, dtype=BF, device="cuda").expand(2, -1, -1, -1))
