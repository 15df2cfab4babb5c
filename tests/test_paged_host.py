"""CPU tests of the paged-cache operators: struct layouts, what the C ABI refuses before
it touches a GPU, and what the Python binding refuses."""
import ctypes

import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import _lib
from differential_attention_fwd_gb300 import build as build_mod

FAKE = 0x10000
INVALID, UNSUPPORTED = _lib.DIFFATTN_ERR_INVALID, _lib.DIFFATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.load()


def rotary_desc(**kw):
    d = _lib.DiffattnRotaryDesc()
    d.B, d.T, d.D, d.H, d.Hk, d.dtype, d.rotary_dim, d.norm, d.eps, d.table_rows = 2, 5, 64, 4, 2, 0, 64, 1, 1e-6, 100
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


def pages(**kw):
    g = _lib.DiffattnPages()
    g.num_pages, g.page_size, g.max_pages, g.block_table_stride = 50, 16, 10, 10
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(g, k)[:] = v
        else:
            setattr(g, k, v)
    return g


def paged_desc(**kw):
    d = _lib.DiffattnPagedDesc()
    d.B, d.H, d.Tq, d.D, d.Dv, d.dtype, d.kv_group = 2, 4, 3, 64, 128, 0, 2
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


def p(i):
    return FAKE * (i + 1)


def rotary(lib, d, x=(1, 1, 1, 1), y=(1, 1, 1, 1), qw=None, kw=None, cos=p(20), sin=p(21)):
    xs = [p(i) if g else None for i, g in enumerate(x)]
    ys = [p(i + 4) if g else None for i, g in enumerate(y)]
    return lib.diffattn_rotary(None if d is None else ctypes.byref(d), *xs, qw, kw, cos, sin, None, *ys, None)


def test_descriptor_layouts():
    # as the header lists the fields, with natural alignment
    R, G, P = _lib.DiffattnRotaryDesc, _lib.DiffattnPages, _lib.DiffattnPagedDesc
    assert ctypes.sizeof(R) == 5 * 8 + 4 * 4 + 4 + 4 + 8 + 2 * 8 + 2 * 8 + 8 * 3 * 8
    assert R.table_rows.offset == 5 * 8 + 6 * 4 and R.q1_grad_stride.offset == ctypes.sizeof(R) - 4 * 3 * 8
    assert ctypes.sizeof(G) == 4 * 8 + 3 * 3 * 8
    assert ctypes.sizeof(P) == 5 * 8 + 2 * 4 + 3 * 3 * 8 + 2 * 8 + 2 * 4 and P.q1_stride.offset == 48


@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0), dict(D=0), dict(D=129), dict(dtype=2), dict(rotary_dim=65),
                                dict(rotary_dim=3), dict(rotary_dim=-2), dict(norm=2), dict(norm=-1), dict(eps=0.0),
                                dict(eps=float("inf")), dict(eps=float("nan")), dict(table_rows=0),
                                dict(pos_stride=(-1, 0)), dict(q_weight_stride=1), dict(k_weight_stride=-64),
                                dict(q1_stride=(-1, 0, 0)), dict(H=0), dict(Hk=0)])
def test_rotary_refusals(lib, kw):
    assert rotary(lib, rotary_desc(**kw)) == INVALID


def test_rotary_argument_refusals(lib):
    assert rotary(lib, None) == INVALID
    assert rotary(lib, rotary_desc(), x=(0, 0, 0, 0), y=(0, 0, 0, 0)) == INVALID
    assert rotary(lib, rotary_desc(), x=(1, 0, 0, 0), y=(0, 0, 0, 0)) == INVALID
    assert rotary(lib, rotary_desc(), x=(1, 0, 0, 0), y=(1, 1, 0, 0)) == INVALID
    assert rotary(lib, rotary_desc(), cos=None) == INVALID
    assert rotary(lib, rotary_desc(norm=0), qw=p(30)) == INVALID
    assert rotary(lib, rotary_desc(B=1 << 20, T=1 << 20)) == UNSUPPORTED
    assert rotary(lib, rotary_desc(B=1, T=(1 << 30) + 1, H=1, Hk=1)) == UNSUPPORTED
    assert rotary(lib, rotary_desc(B=1 << 15, T=1 << 15, H=300)) == UNSUPPORTED
    assert rotary(lib, rotary_desc(H=40000)) == UNSUPPORTED


def test_rotary_backward_refusals(lib):
    def bwd(d, dys=(1, 1, 1, 1), dqw=None, dkw=None, ws=p(40), n=1 << 30, x=(1, 1, 1, 1)):
        xs = [p(i) if g else None for i, g in enumerate(x)]
        return lib.diffattn_rotary_bwd(ctypes.byref(d), *xs, None, None, p(20), p(21), None,
                                       *[p(8 + i) if g else None for i, g in enumerate(dys)],
                                       *[p(12 + i) if g else None for i, g in enumerate(x)], dqw, dkw, ws, n, None)
    need = lib.diffattn_rotary_bwd_workspace_bytes(ctypes.byref(rotary_desc()))
    assert need > 0
    assert lib.diffattn_rotary_bwd_workspace_bytes(ctypes.byref(rotary_desc(D=0))) == 0
    assert lib.diffattn_rotary_bwd_workspace_bytes(None) == 0
    assert bwd(rotary_desc(), dys=(1, 1, 1, 0)) == INVALID
    assert bwd(rotary_desc(), x=(1, 0, 0, 0)) == INVALID
    assert bwd(rotary_desc(q2_grad_stride=(0, -1, 0))) == INVALID
    assert bwd(rotary_desc(norm=0), dqw=p(30)) == INVALID
    assert bwd(rotary_desc(), ws=None) == INVALID
    assert bwd(rotary_desc(), ws=p(40) + 8) == INVALID
    assert bwd(rotary_desc(), n=need - 1) == INVALID
    assert bwd(rotary_desc(), x=(1, 0, 1, 0), dys=(1, 0, 1, 0), dkw=p(31)) == INVALID


@pytest.mark.parametrize("kw", [dict(H=-2), dict(Hk=-2), dict(H=-1, Hk=-1), dict(H=-(1 << 40))])
def test_rotary_negative_head_counts(lib, kw):
    """A negative count is refused where its tensors are left out too: the backward's workspace goes
    by both.  (A workspace of one byte, so that no call can get as far as a GPU.)"""
    for T in (5, 1 << 20):
        d = rotary_desc(B=1, T=T, **kw)
        for x in ((0, 1, 0, 0), (0, 1, 0, 1), (1, 0, 1, 0)):
            assert rotary(lib, d, x=x, y=x) == INVALID, (kw, T, x)
            xs, ys, gs = ([p(j + i) if g else None for i, g in enumerate(x)] for j in (0, 4, 8))
            assert lib.diffattn_rotary_bwd(ctypes.byref(d), *xs, None, None, p(20), p(21), None, *gs, *ys, None, None,
                                           p(40), 1, None) == INVALID
        assert lib.diffattn_rotary_bwd_workspace_bytes(ctypes.byref(d)) == 0


def test_append_refusals(lib):
    def append(d=None, Dv=128, vs=(0, 0, 0), g=None, k2=p(1), k2c=p(6), **miss):
        a = dict(k1=p(0), v=p(2), lens=p(3), table=p(4), k1c=p(5), vc=p(7), kw=None)
        a.update(miss)
        d, g = d or rotary_desc(), g or pages()
        return lib.diffattn_paged_append(ctypes.byref(d), Dv, (ctypes.c_int64 * 3)(*vs), ctypes.byref(g), a["k1"], k2,
                                         a["v"], a["kw"], p(20), p(21), None, a["lens"], None, a["table"], a["k1c"],
                                         k2c, a["vc"], None)
    for miss in ("k1", "v", "lens", "table", "k1c", "vc"):
        assert append(**{miss: None}) == INVALID
    assert append(k2=None) == INVALID and append(k2c=None) == INVALID
    assert append(k2c=p(5)) == INVALID                       # two tensors of keys into one cache
    assert append(Dv=257) == INVALID and append(Dv=-1) == INVALID and append(vs=(0, -1, 0)) == INVALID
    assert append(d=rotary_desc(Hk=0)) == INVALID and append(d=rotary_desc(T=0)) == INVALID
    assert append(d=rotary_desc(norm=0), kw=p(30)) == INVALID
    for kw in (dict(num_pages=0), dict(page_size=0), dict(max_pages=0), dict(block_table_stride=-1),
               dict(k1_stride=(-1, 0, 0)), dict(v_stride=(0, 0, -1))):
        assert append(g=pages(**kw)) == INVALID
    assert append(g=pages(page_size=1 << 21)) == UNSUPPORTED
    assert append(d=rotary_desc(Hk=30000)) == UNSUPPORTED
    # one place for two tokens, and one cache twice
    k, v = (16 * 128, 16 * 64, 64), (16 * 256, 16 * 128, 128)
    for i in range(3):
        for name, s in (("k1_stride", k), ("k2_stride", k), ("v_stride", v)):
            good = dict(k1_stride=k, k2_stride=k, v_stride=v)
            good[name] = tuple(0 if j == i else s[j] for j in range(3))
            assert append(g=pages(**good)) == INVALID, (name, i)
    good = dict(k1_stride=k, k2_stride=k, v_stride=v)
    assert append(g=pages(**good), vc=p(5)) == INVALID and append(g=pages(**good), vc=p(6)) == INVALID


def decode(lib, d=None, g=None, ws=p(40), n=1 << 30, mask=None, lam=0.5, epi=None, **miss):
    a = dict(q1=p(0), k1=p(1), q2=p(2), k2=p(3), v=p(4), table=p(5), lens=p(6), out=p(7))
    a.update(miss)
    d, g = d or paged_desc(), g or pages()
    return lib.diffattn_paged_decode(ctypes.byref(d), ctypes.byref(g), a["q1"], a["k1"], a["q2"], a["k2"], a["v"],
                                     a["table"], a["lens"], None, mask, lam, None,
                                     None if epi is None else ctypes.byref(epi), a["out"], ws, n, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(H=0), dict(Tq=0), dict(D=0), dict(D=129), dict(Dv=257), dict(Dv=-1),
                                dict(dtype=3), dict(kv_group=3), dict(kv_group=-1), dict(q1_stride=(-1, 0, 0)),
                                dict(o_stride=(0, 0, -1)), dict(mask_stride=(0, -1)), dict(zero_rest=2), dict(zero_rest=-1),
                                dict(reserved=1)])
def test_decode_refusals(lib, kw):
    assert lib.diffattn_paged_workspace_bytes(ctypes.byref(paged_desc(**kw)), ctypes.byref(pages())) == 0
    assert decode(lib, paged_desc(**kw)) == INVALID


def test_decode_argument_refusals(lib):
    for miss in ("q1", "k1", "q2", "k2", "v", "table", "lens", "out"):
        assert decode(lib, **{miss: None}) == INVALID
    assert decode(lib, ws=None) == INVALID and decode(lib, ws=p(40) + 8) == INVALID
    assert decode(lib, lam=float("nan")) == INVALID
    assert decode(lib, epi=_lib.DiffattnEpilogue(norm=7, eps=1e-5, out_scale=1.0)) == INVALID
    assert decode(lib, paged_desc(Tq=65), mask=p(8)) == INVALID
    assert decode(lib, paged_desc(Tq=1025)) == UNSUPPORTED
    assert decode(lib, g=pages(num_pages=1 << 31)) == UNSUPPORTED
    for o in ((0, 128, 512), (4 * 3 * 128, 0, 128), (4 * 3 * 128, 128, 0)):
        assert decode(lib, paged_desc(o_stride=o)) == INVALID
    assert lib.diffattn_paged_workspace_bytes(ctypes.byref(paged_desc()), ctypes.byref(pages())) > 0


def test_device_error_has_a_text(lib):
    assert lib.diffattn_strerror(_lib.DIFFATTN_ERR_INDEX) not in (lib.diffattn_strerror(0), lib.diffattn_strerror(99))


def test_tables_are_exact_at_far_positions():
    cos, sin = da.rotary_tables(200001, 8)
    assert cos.dtype == torch.float32 and cos.shape == (200001, 4)
    import math
    for pos in (0, 1, 65537, 200000):
        for i in range(4):
            a = pos * 10000.0 ** (-2 * i / 8)
            # half a step of a float32 below 1, and the float64 angle's own error
            assert abs(float(cos[pos, i]) - math.cos(a)) <= 2.0 ** -25 + 1e-10
            assert abs(float(sin[pos, i]) - math.sin(a)) <= 2.0 ** -25 + 1e-10
    for bad in ((0, 8), (5, 3), (5, 0)):
        with pytest.raises(ValueError):
            da.rotary_tables(*bad)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64)
    c = torch.zeros(4, 2, 16, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="no CPU path"):
        da.qk_norm_rotary(x, x, x, x, None, None)
    with pytest.raises(ValueError, match="no CPU path"):
        da.paged_cache_append(x, x, x, c, c, c, i, n)
    with pytest.raises(ValueError, match="no CPU path"):
        da.differential_attention_paged(x, c, x, c, c, i, n, 0.5)
    with pytest.raises(TypeError):
        da.differential_attention_tree(x, c, x, c, c, i, n, None, 0.5)
    with pytest.raises(ValueError):
        da.qk_norm_rotary(None, None, None, None, None, None)
