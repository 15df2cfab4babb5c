"""CPU tests of a cross-attention block's operators: struct layouts, what the C ABI refuses
before it touches a GPU, what the Python binding refuses, and the reference's gradients
against differences."""
import ctypes

import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import _lib
from differential_attention_fwd_gb300 import build as build_mod
from tests import block_reference as ref

FAKE = 0x10000
INVALID, UNSUPPORTED = _lib.DIFFATTN_ERR_INVALID, _lib.DIFFATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def p(i):
    return FAKE * (i + 1)


def fill(d, **kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


def differences(f, x, dy, h=1e-6):
    """Gradient of (f(x) dy).sum() by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = (f() * dy).sum()
        flat[i] = keep - h
        out[i] = (up - (f() * dy).sum()) / (2 * h)
        flat[i] = keep
    return g


# ------------------------------------------------------------------ head norm
def norm_desc(**kw):
    d = _lib.DiffattnNormDesc()
    d.B, d.H, d.T, d.C, d.dtype, d.norm, d.eps, d.out_scale = 2, 3, 5, 128, 0, 1, 1e-6, 1.0
    for f in ("x_stride", "y_stride", "dy_stride", "dx_stride"):
        getattr(d, f)[:] = (3 * 5 * 128, 5 * 128, 128)
    return fill(d, **kw)


def test_norm_descriptor_layout():
    N = _lib.DiffattnNormDesc
    assert ctypes.sizeof(N) == 4 * 8 + 4 * 4 + 4 * 3 * 8 and N.x_stride.offset == 48


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=0), dict(T=0), dict(C=0), dict(C=257), dict(dtype=2), dict(norm=0),
                                dict(norm=3), dict(eps=0.0), dict(eps=float("nan")), dict(out_scale=float("inf")),
                                dict(x_stride=(-1, 0, 0)), dict(dy_stride=(0, -1, 0)), dict(y_stride=(0, 640, 128)),
                                dict(y_stride=(1920, 640, 0))])
def test_norm_refusals(lib, kw):
    assert lib.diffattn_head_norm(ctypes.byref(norm_desc(**kw)), p(0), None, None, p(1), None) == INVALID


def test_norm_argument_refusals(lib):
    def bwd(d=None, x=p(0), dy=p(1), dx=p(2), dw=p(3), db=None, ws=p(4), n=1 << 30):
        return lib.diffattn_head_norm_bwd(ctypes.byref(d or norm_desc()), x, None, dy, dx, dw, db, ws, n, None)
    d = norm_desc()
    assert lib.diffattn_head_norm(None, p(0), None, None, p(1), None) == INVALID
    assert lib.diffattn_head_norm(ctypes.byref(d), None, None, None, p(1), None) == INVALID
    assert lib.diffattn_head_norm(ctypes.byref(d), p(0), None, None, None, None) == INVALID
    for big in (dict(H=65536), dict(T=(1 << 30) + 1), dict(B=1 << 16, T=1 << 16)):
        assert lib.diffattn_head_norm(ctypes.byref(norm_desc(**big)), p(0), None, None, p(1), None) == UNSUPPORTED
    need = lib.diffattn_head_norm_bwd_workspace_bytes(ctypes.byref(d))
    assert need > 0 and lib.diffattn_head_norm_bwd_workspace_bytes(None) == 0
    assert lib.diffattn_head_norm_bwd_workspace_bytes(ctypes.byref(norm_desc(C=0))) == 0
    assert bwd(x=None) == INVALID and bwd(dy=None) == INVALID and bwd(dx=None, dw=None) == INVALID
    assert bwd(ws=None) == INVALID and bwd(ws=p(4) + 8) == INVALID and bwd(n=need - 1) == INVALID
    assert bwd(d=norm_desc(dx_stride=(0, 640, 128))) == INVALID


@pytest.mark.parametrize("group", [False, True])
def test_norm_reference_gradients(group):
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(2, 2, 3, 5, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(2, 5, generator=g, dtype=torch.float64) for _ in range(2))
    f = lambda: ref.head_norm(x, group, 1e-3, w, b, 0.3)[0]         # noqa: E731
    dx, dw, db = ref.head_norm_backward(x, group, 1e-3, w, 0.3, dy)
    # central differences with h = 1e-6: h^2 of the third derivative, and 2^-53 / h of the values
    for t, want in ((x, dx), (w, dw), (b, db)):
        torch.testing.assert_close(differences(f, t, dy), want, rtol=0, atol=1e-7)


# ------------------------------------------------------------------ cross attention
def cross_desc(**kw):
    d = _lib.DiffattnCrossDesc()
    d.B, d.H, d.Tq, d.Tk, d.D, d.Dv, d.dtype, d.kv_group = 2, 4, 5, 7, 64, 128, 0, 2
    for f, rows, width in (("q1_stride", 5, 64), ("q2_stride", 5, 64), ("k1_stride", 7, 64), ("k2_stride", 7, 64),
                           ("v_stride", 7, 128), ("o_stride", 5, 128), ("dout_stride", 5, 128)):
        heads = 4 if rows == 5 else 2
        getattr(d, f)[:] = (heads * rows * width, rows * width, width)
    return fill(d, **kw)


def cross_fwd(lib, d=None, lam=0.5, epi=None, out2=None, lse=None, ws=p(40), n=1 << 30, **miss):
    a = dict(q1=p(0), k1=p(1), q2=p(2), k2=p(3), v=p(4), out=p(5))
    a.update(miss)
    return lib.diffattn_cross_fwd(ctypes.byref(d or cross_desc()), a["q1"], a["k1"], a["q2"], a["k2"], a["v"], None, lam, None,
                                  None if epi is None else ctypes.byref(epi), a["out"], out2, lse, ws, n, None)


def cross_bwd(lib, d=None, lam=0.5, ws=p(40), n=1 << 30, **other):
    a = dict(q1=p(0), k1=p(1), q2=p(2), k2=p(3), v=p(4), out=p(5), out2=p(6), lse=p(7), dout=p(8), dq1=p(9), dk1=p(10),
             dq2=p(11), dk2=p(12), dv=p(13), dlam=p(14))
    a.update(other)
    return lib.diffattn_cross_bwd(ctypes.byref(d or cross_desc()), a["q1"], a["k1"], a["q2"], a["k2"], a["v"], None, lam, None,
                                  a["out"], a["out2"], a["lse"], a["dout"], a["dq1"], a["dk1"], a["dq2"], a["dk2"], a["dv"],
                                  a["dlam"], ws, n, None)


def test_cross_descriptor_layout():
    C = _lib.DiffattnCrossDesc
    assert ctypes.sizeof(C) == 6 * 8 + 4 * 4 + 7 * 3 * 8 and C.q1_stride.offset == 64


BAD_CROSS = [dict(lambda_dtype=2), dict(reserved=1), dict(B=0), dict(H=0), dict(Tq=0), dict(Tk=0), dict(D=0), dict(D=129), dict(Dv=-1), dict(Dv=257), dict(dtype=2),
             dict(kv_group=-1), dict(kv_group=3), dict(q1_stride=(-1, 0, 0)), dict(k2_stride=(0, -1, 0)), dict(v_stride=(0, 0, -1)),
             dict(dout_stride=(-1, 0, 0))]


@pytest.mark.parametrize("kw", BAD_CROSS)
def test_cross_refusals(lib, kw):
    d = cross_desc(**kw)
    assert cross_fwd(lib, d) == INVALID and cross_bwd(lib, d) == INVALID
    assert lib.diffattn_cross_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.diffattn_cross_bwd_workspace_bytes(ctypes.byref(d)) == 0


def test_cross_argument_refusals(lib):
    for miss in ("q1", "k1", "q2", "k2", "v", "out"):
        assert cross_fwd(lib, **{miss: None}) == INVALID and cross_bwd(lib, **{miss: None}) == INVALID
    for miss in ("out2", "lse", "dout", "dk1", "dv"):
        assert cross_bwd(lib, **{miss: None}) == INVALID
    assert cross_bwd(lib, dk2=None) == INVALID                          # two key tensors, one gradient
    assert cross_bwd(lib, dq1=None, dq2=None, dk1=None, dk2=None, dv=None, dlam=None) == INVALID
    assert cross_fwd(lib, out2=p(6)) == INVALID and cross_fwd(lib, lse=p(7)) == INVALID
    assert cross_fwd(lib, lam=float("nan")) == INVALID and cross_bwd(lib, lam=float("inf")) == INVALID
    for epi in (_lib.DiffattnEpilogue(norm=1, eps=1e-5, out_scale=1.0), _lib.DiffattnEpilogue(out_scale=0.5)):
        assert cross_fwd(lib, epi=epi, out2=p(6), lse=p(7)) == INVALID
    assert cross_fwd(lib, epi=_lib.DiffattnEpilogue(norm=9, eps=1e-5, out_scale=1.0)) == INVALID
    assert cross_fwd(lib, epi=_lib.DiffattnEpilogue(weight=p(50), out_scale=1.0)) == INVALID       # of no norm
    assert cross_fwd(lib, cross_desc(o_stride=(0, 640, 128))) == INVALID
    need = lib.diffattn_cross_bwd_workspace_bytes(ctypes.byref(cross_desc()))
    assert need >= 2 * 4 * 5 * 16
    for f in (cross_fwd, cross_bwd):
        assert f(lib, ws=None) == INVALID and f(lib, ws=p(40) + 8) == INVALID and f(lib, n=0) == INVALID
    assert cross_bwd(lib, n=need - 1) == INVALID
    for big in (dict(Tq=1 << 31), dict(Tk=1 << 31), dict(B=1 << 20, Tq=1 << 18)):
        assert cross_fwd(lib, cross_desc(**big)) == UNSUPPORTED


def test_cross_rests_refusals(lib):
    def fwd(d=None, out2=p(6), lse=p(7), rests=p(8)):
        return lib.diffattn_cross_fwd_ex(ctypes.byref(d or cross_desc()), *map(p, range(5)), None, 0.5, None, None, p(5), out2, lse,
                                         rests, p(40), 1 << 30, None)

    def bwd(d=None, rests=p(8)):
        return lib.diffattn_cross_bwd_ex(ctypes.byref(d or cross_desc()), *map(p, range(5)), None, 0.5, None, p(5), p(6), p(7), rests,
                                         p(9), *map(p, range(10, 15)), p(15), p(40), 1 << 30, None)
    assert fwd(out2=None, lse=None) == INVALID                         # nothing to leave a rest of
    for kw in (dict(rests=p(8) + 8), dict(d=cross_desc(dtype=1))):
        assert fwd(**kw) == INVALID and bwd(**kw) == INVALID


@pytest.mark.parametrize("lens", [[4, 2], [3, 0]])
def test_cross_reference_gradients(lens):
    g = torch.Generator().manual_seed(1)
    q1, q2 = (torch.randn(2, 4, 3, 5, generator=g, dtype=torch.float64) for _ in range(2))
    k1, k2 = (torch.randn(2, 2, 4, 5, generator=g, dtype=torch.float64) for _ in range(2))
    v, do = torch.randn(2, 2, 4, 6, generator=g, dtype=torch.float64), torch.randn(2, 4, 3, 6, generator=g, dtype=torch.float64)
    x = [q1, k1, q2, k2, v]
    lam = torch.tensor(0.7, dtype=torch.float64)
    f = lambda: ref.Cross(*x, lam, lens, ref.U).o                      # noqa: E731
    got = ref.Cross(*x, lam, lens, ref.U).backward(do)
    for t, name in list(zip(x, ("q1", "k1", "q2", "k2", "v"))) + [(lam, "lam")]:
        torch.testing.assert_close(differences(f, t, do), got[name][0], rtol=0, atol=1e-7)
    k2.copy_(k1)                                                       # one key tensor: moved together
    x[3] = k1
    torch.testing.assert_close(differences(f, k1, do), ref.Cross(*x, lam, lens, ref.U).backward(do)["k"][0], rtol=0, atol=1e-7)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="no CPU path"):
        da.differential_cross_attention(x, x, x, x, x, 0.5)
    with pytest.raises(ValueError, match="no CPU path"):
        da.differential_head_norm(x)


# ------------------------------------------------------------------ positions with several axes
def test_axes_layout_and_refusals(lib):
    assert ctypes.sizeof(_lib.DiffattnAxes) == 4 * 6 + 8

    def axes(n, *pairs, reserved=0, stride=1):
        a = _lib.DiffattnAxes()
        a.n, a.reserved, a.pos_stride = n, reserved, stride
        for i, v in enumerate(pairs):
            a.pairs[i] = v
        return a

    def rotary(a, R=64, pos=p(30)):
        d = _lib.DiffattnRotaryDesc()
        d.B, d.T, d.D, d.H, d.Hk, d.dtype, d.rotary_dim, d.norm, d.eps, d.table_rows = 2, 5, 64, 4, 2, 0, R, 1, 1e-6, 100
        return [lib.diffattn_rotary_axes(ctypes.byref(d), ctypes.byref(a), p(0), None, None, None, None, None, p(20), p(21), pos,
                                         p(4), None, None, None, None),
                lib.diffattn_rotary_axes_bwd(ctypes.byref(d), ctypes.byref(a), p(0), None, None, None, None, None, p(20), p(21), pos,
                                             p(8), None, None, None, p(4), None, None, None, None, None, p(40), 1 << 30, None)]
    for a in (axes(0), axes(5, 8, 8, 8, 8), axes(2, 16, 15), axes(2, 16, 17), axes(2, 32, 0), axes(2, -1, 33), axes(1, 33),
              axes(1, 32, reserved=1), axes(1, 32, stride=-1), axes(-1)):
        assert rotary(a) == [INVALID, INVALID]
    assert rotary(axes(1, 32), pos=None) == [INVALID, INVALID]
    assert rotary(axes(1, 1), R=0) == [INVALID, INVALID]


def test_tables_of_sections():
    cos, sin = da.rotary_tables(300, 24, sections=(2, 4, 6))
    f = [100.0 ** -i for i in range(2)] + [10.0 ** -i for i in range(4)] + [10000.0 ** (-i / 6) for i in range(6)]
    a = torch.arange(300, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    # half a step of a float32 below 1, and the float64 angles' own errors
    assert ((cos.double() - a.cos()).abs() <= 2.0 ** -25 + 1e-11).all() and ((sin.double() - a.sin()).abs() <= 2.0 ** -25 + 1e-11).all()
    one = da.rotary_tables(50, 16, sections=(8,))
    assert all(torch.equal(x, y) for x, y in zip(one, da.rotary_tables(50, 16)))
    for bad in ((), (4, 5), (8, 0), (12,)):
        with pytest.raises(ValueError):
            da.rotary_tables(50, 16, sections=bad)
