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


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="no CPU path"):
        da.differential_head_norm(x)
