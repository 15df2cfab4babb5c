"""GPU tests of differential attention over a paged cache on the paths that a call's size or
layout chooses, against float64: scores of any size, many short sequences, long chunks,
queries and outputs that the wide copies do not take."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import paged_reference as ref
from tests.test_gpu_paged import HEADS, LAM, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _clean():
    da.get_device_error()
    yield
    assert da.get_device_error() == 0


def put_keys(pb):
    """Writes pb.k1 and pb.k2 into the caches again."""
    for b in range(len(pb.lens)):
        for cache, rows in ((0, pb.k1[b]), (1, pb.k2[b])):
            for t in range(0, rows.shape[1], pb.page):
                part = rows[:, t:t + pb.page]
                pb.caches[cache][int(pb.table[b, t // pb.page]), :, :part.shape[1]] = part.cuda()


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,tree", [(1, False), (6, True), (20, False), (40, True)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [12, 15, 16, 17, 53])
@pytest.mark.parametrize("qf,kf", [(1.0, 1.0), (1 + 45 / 128, 1 + 91 / 128)])
def test_scores_of_any_size(head, Tq, tree, sign, size, qf, kf):
    """Queries of qf 2^size and keys of sign kf 2^size or twice that: of the two scores, 2^(2 size) and
    more apart and both exact, the higher one's keys share a weight of 1 and the others have none,
    exactly (from 2^24 on, where an exponential is 0).  A score times the scale is a float32 for the
    first pair of factors and not for the second."""
    pb = Problem(*head, 2, 1, Tq, [300, 33, 900], 16, tree=tree)
    g = torch.Generator().manual_seed(size)
    pb.q1.fill_(qf * 2.0 ** size)
    pb.q2.fill_(qf * 2.0 ** size)
    for ks in (pb.k1,) if pb.shared else (pb.k1, pb.k2):
        for k in ks:
            level = 1 + torch.randint(0, 2, (k.shape[0], k.shape[1], 1), generator=g)
            k.copy_((sign * kf * 2.0 ** size * level).expand(k.shape))
    put_keys(pb)
    out = pb.run().cpu().double()
    h = ref.half_step(pb.dtype)
    for b, head_, o, _ in pb.want():
        # weights of 0 and 1: what is left is the sums (n terms), a division and a few roundings of
        # the means of |v|, at most max|v|, and the result's
        n = pb.lens[b] + Tq
        top = (1 + LAM) * pb.v[b][0].double().abs().amax(0)
        got = out[b, head_, :o.shape[0]]
        assert torch.isfinite(got).all(), (b, head_)
        over = (got - o).abs() - (h * o.abs() + (1 + h) * ref.U * (n + 8) * top)
        assert over.max() <= 0, (b, head_)


def finite_rows(q1, k1, q2, k2, v, seen, lam, dtype):
    """ref.attention_rows (the same formulas) for values that are finite, by products of matrices."""
    n, D = k1.shape
    o, size, e = 0, 0, 0
    for q, k, f in ((q1, k1, 1.0), (q2, k2, -lam)):
        a = torch.softmax((q @ k.T / D ** 0.5).masked_fill(~seen, float("-inf")), -1)
        o, size = o + f * (a @ v), size + abs(f) * (a @ v.abs())
        z = (q.abs() @ k.abs().T / D ** 0.5).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
        e = torch.maximum(torch.as_tensor(e, dtype=v.dtype), ref.U * (n + 2 * D * z + 2 * z + 16))
    h = ref.half_step(dtype)
    parts = h * h if dtype == torch.bfloat16 else 0.0
    return o, (1 + h) * (2 * e + 4 * ref.U + parts) * size + h * o.abs()


def some(pb, picks, lam=LAM):
    """(b, h, o, bound) of some sequences' heads, of those with new tokens."""
    for b, h in picks:
        t = pb.new[b]
        if t == 0:
            continue
        seen = ref.visible(pb.lens[b], t, None if pb.tree is None else pb.tree[b, :t, :t])
        hk = h // (pb.H // pb.Hk)
        yield b, h, *finite_rows(pb.q1[b, h, :t].double().cpu(), pb.k1[b][hk].double(), pb.q2[b, h, :t].double().cpu(),
                                 pb.k2[b][hk].double(), pb.v[b][hk].double(), seen, lam, pb.dtype)


def check_some(pb, out, picks, what, lam=LAM):
    out = out.cpu().double()
    for b, h, o, bound in some(pb, picks, lam):
        got = out[b, h, :o.shape[0]]
        assert torch.isfinite(got).all(), f"{what} b={b} h={h}"
        over = ((got - o).abs() - bound).max()
        assert over <= 0, f"{what} b={b} h={h}: {float(over)} over the bound"


# ---------------------------------------------------------------------------
# Many units of few rows: a warp is a worker by itself (up to 8 rows a key/value head at Q/K
# width 64, 4 at 128; two units for three of the GPU's warps).
# ---------------------------------------------------------------------------
BF16 = HEADS[:4]
MANY_HK = 8


def many(head, rows, group=1, tree=False, lens=None, new=None, **kw):
    """640 units or more.  Most sequences are short; some are long enough to be split over warps."""
    Tq = rows // group
    lens = lens or [(53 * b) % 200 for b in range(80)]
    lens[3], lens[40], lens[41], lens[79] = 2100, 0, 700, 1300
    assert 2 * len(lens) * MANY_HK >= 8 * torch.cuda.get_device_properties(0).multi_processor_count
    new = new or [Tq if b % 7 else 1 + b % Tq for b in range(len(lens))]
    return Problem(*head, MANY_HK * group, MANY_HK, Tq, lens, 16, new=new, tree=tree, **kw)


def picks(pb):
    """The special sequences and some others, a head each or two."""
    return [(b, (3 * b + i) % pb.H) for b in (0, 1, 3, 8, 14, 21, 40, 41, 57, 62, 77, 79) for i in (0, pb.H - 1)]


def rows_of(head):
    return (1, 2, 4, 8) if head[1] == 64 else (1, 2, 4)


def misaligned_out(pb):
    """(buffer of sevens, output in it): rows of an odd stride that start at an odd element."""
    buf = torch.full((len(pb.lens), pb.H, pb.Tq, pb.Dv + 3), 7.0, dtype=pb.dtype, device="cuda")
    return buf, buf[..., 1:1 + pb.Dv]


def check_around(pb, buf, out):
    assert (buf[..., 0] == 7).all() and (buf[..., 1 + pb.Dv:] == 7).all()
    for b, t in enumerate(pb.new):
        assert (out[b, :, t:] == 7).all()


@pytest.mark.parametrize("head", BF16)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("group", [1, 2])
def test_many_units(head, tree, group):
    for rows in rows_of(head):
        if rows < group:
            continue
        pb = many(head, rows, group, tree)
        check_some(pb, pb.run(), picks(pb), f"{rows} rows")


@pytest.mark.parametrize("head", BF16)
@pytest.mark.parametrize("norm", ["rms", "group", None])
@pytest.mark.parametrize("odd", [False, True])
def test_many_units_epilogue_and_outputs(head, norm, odd):
    g = torch.Generator().manual_seed(2)
    for rows, group in ((1, 1), (rows_of(head)[-1], 2)):
        pb = many(head, rows, group)
        w, bias = (torch.randn(pb.H, pb.Dv, generator=g) for _ in range(2))
        buf, place = misaligned_out(pb)
        out = pb.run(norm=norm, norm_eps=1e-5, norm_weight=w.cuda(), norm_bias=bias.cuda(), out_scale=0.2,
                     out=place if odd else None)
        if odd:
            check_around(pb, buf, out)
        out = out.cpu().double()
        for b, h, o, bound in some(pb, picks(pb)):
            y, tol = ref.epilogue(o, bound, norm, 1e-5, w[h].double(), bias[h].double(), 0.2, pb.dtype)
            assert ((out[b, h, :o.shape[0]] - y).abs() <= tol).all(), f"{rows} rows b={b} h={h}"


@pytest.mark.parametrize("head", BF16)
@pytest.mark.parametrize("slope,spikes", [(0.04, False), (-0.04, False), (0.01, True), (0.0, True)])
def test_many_units_moving_maximum(head, slope, spikes):
    for rows in (1, rows_of(head)[-1]):
        pb = many(head, rows, slope=slope / 3, spikes=spikes, tree=rows > 1 and spikes)
        check_some(pb, pb.run(), picks(pb), f"{rows} rows")


@pytest.mark.parametrize("head", BF16)
def test_many_units_scores_of_any_size(head):
    """As test_scores_of_any_size."""
    for size in (12, 17, 53):
        pb = many(head, rows_of(head)[-1])
        g = torch.Generator().manual_seed(size)
        pb.q1.fill_(1.3515625 * 2.0 ** size)
        pb.q2.fill_(1.3515625 * 2.0 ** size)
        for ks in (pb.k1,) if pb.shared else (pb.k1, pb.k2):
            for k in ks:
                level = 1 + torch.randint(0, 2, (k.shape[0], k.shape[1], 1), generator=g)
                k.copy_((-1.7109375 * 2.0 ** size * level).expand(k.shape))
        put_keys(pb)
        out, h = pb.run().cpu().double(), ref.half_step(pb.dtype)
        for b, head_, o, _ in some(pb, picks(pb)):
            top = (1 + LAM) * pb.v[b][head_].double().abs().amax(0)
            over = (out[b, head_, :o.shape[0]] - o).abs() - (h * o.abs() + (1 + h) * ref.U * (pb.lens[b] + pb.Tq + 8) * top)
            assert over.max() <= 0, (size, b, head_)


@pytest.mark.parametrize("head", BF16)
def test_many_units_values_that_are_not_finite(head):
    """In a visible value: its column is NaN for that head.  In a drafted token's: for the rows that
    see it.  In its keys: those rows, whole."""
    rows = rows_of(head)[-1]
    pb = many(head, rows, tree=True, new=[rows] * 80)
    clean = pb.run()
    check_some(pb, clean, picks(pb), "clean")
    for b, at in ((8, 5), (3, 1999), (41, pb.lens[41] + 1), (0, 1), (57, pb.lens[57])):
        pg, row = int(pb.table[b, at // 16]), at % 16
        sees = torch.ones(rows, dtype=torch.bool) if at < pb.lens[b] else pb.tree[b, :, at - pb.lens[b]]
        assert sees.any()
        for value in (float("nan"), float("inf"), -float("inf")):
            old = pb.caches[2][pg, 2, row, 3].clone()
            pb.caches[2][pg, 2, row, 3] = value
            out = pb.run()
            pb.caches[2][pg, 2, row, 3] = old
            assert not torch.isfinite(out[b, 2, sees.cuda(), 3]).any(), (b, at, value)
            assert torch.isfinite(out[b, 2, ~sees.cuda(), 3]).all()
            out[b, 2, sees.cuda(), 3] = clean[b, 2, sees.cuda(), 3]
            check_some(pb, out, [(b, 2), (b, 3), (40, 2)], f"{value} at {at} of {b}")
    b = 57
    hidden = 1
    at, sees = pb.lens[b] + hidden, pb.tree[b, :, hidden].cuda()
    pg, row = int(pb.table[b, at // 16]), at % 16
    pb.caches[0][pg, 2, row] = float("nan")
    out = pb.run()
    assert torch.isnan(out[b, 2, sees]).all()
    out[b, 2, sees] = clean[b, 2, sees]
    check_some(pb, out, [(b, 2), (b, 1)], "hidden key")


@pytest.mark.parametrize("head", BF16)
def test_many_units_rows_that_see_nothing_and_branches_that_cancel(head):
    rows = rows_of(head)[-1]
    pb = many(head, rows, tree=True, new=[rows] * 80)
    pb.tree[40, 0] = False                          # sequence 40 has no cached token
    out = pb.run()
    assert torch.count_nonzero(out[40, :, 0]) == 0 and torch.isfinite(out).all()
    out = pb.run(norm="rms", norm_bias=torch.ones(pb.H, pb.Dv, device="cuda"), out_scale=0.5)
    assert (out[40, :, 0] == 0.5).all()
    pb = many(head, rows)
    for lam in (-0.7, 0.0, torch.tensor(0.6, device="cuda")):
        check_some(pb, pb.run(lam=lam), picks(pb)[::3], f"lambda {lam}", float(lam))
    pb.q2, pb.shared = pb.q1, True
    assert torch.count_nonzero(pb.run(lam=1.0)) == 0


@pytest.mark.parametrize("head", BF16)
def test_many_units_out_of_range(head):
    rows = rows_of(head)[-1]
    pb = many(head, rows)
    good = pb.run()
    k1, k2, v = pb.caches
    for what, b in (("length", 8), ("negative", 41), ("page", 3), ("low page", 79), ("count", 57)):
        table, ln, new = pb.table.clone(), torch.tensor(pb.lens, dtype=torch.int32), torch.tensor(pb.new, dtype=torch.int32)
        if what == "length":
            ln[b] = table.shape[1] * 16
        elif what == "negative":
            ln[b] = -1
        elif what == "page":
            table[b, 60] = k1.shape[0]
        elif what == "low page":
            table[b, 0] = -1
        else:
            new[b] = pb.Tq + 1
        out = da.differential_attention_paged(pb.q1, k1, pb.q2, k1 if pb.shared else k2, v, table.cuda(), ln.cuda(), LAM,
                                              q_lengths=new.cuda())
        assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX, what
        asked = pb.Tq if int(new[b]) > pb.Tq or what in ("length", "negative") else int(new[b])
        assert torch.isnan(out[b, :, :asked]).all(), what
        # (the division of the work follows the lengths, so the others are compared to the bound)
        rest = [i for i in range(80) if i != b]
        assert torch.isfinite(out[rest]).all(), what
        check_some(pb, out, [(i, h) for i, h in picks(pb) if i != b], what)
    assert torch.equal(good, pb.run())


@pytest.mark.parametrize("head", BF16)
@pytest.mark.parametrize("active", [1, 3, 40])
def test_many_places_few_of_them_active(head, active):
    """The host sees many units, and the device finds few: a block is a worker, and the merging pass
    reads words of workers that there are not."""
    rows = rows_of(head)[-1]
    lens = [0] * 160
    new = [0] * 160
    for i in range(active):
        lens[(i * 37 + 5) % 160], new[(i * 37 + 5) % 160] = 900 + 13 * i if active < 10 else 70 + i, rows - i % 2
    pb = Problem(*head, MANY_HK, MANY_HK, rows, lens, 16, new=new)
    for again in range(2):                          # and the workspace as the last call left it
        out = pb.run()
        check_some(pb, out, [(b, (b + i) % 8) for b in range(160) if new[b] for i in range(0, 8, 3)][:40], f"{active} active")
        for b, t in enumerate(new):
            assert torch.count_nonzero(out[b, :, t:]) == 0


# ---------------------------------------------------------------------------
# chunks of a prefill, up to the most tokens that a call takes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,H,Hk,page", [(131, 2, 1, 16), (192, 3, 3, 32), (257, 4, 1, 16), (500, 2, 2, 48), (777, 2, 1, 64),
                                          (1024, 2, 1, 128)])
def test_long_chunks(head, Tq, H, Hk, page):
    pb = Problem(*head, H, Hk, Tq, [0, 37, 300, 64, 5], page, new=[Tq, Tq - 1, Tq // 2 + 1, 1, 0])
    out = pb.run()
    check_some(pb, out, [(b, h) for b in range(5) for h in (0, H - 1)], f"Tq={Tq}")
    for b, t in enumerate(pb.new):
        assert torch.count_nonzero(out[b, :, t:]) == 0


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("before", [0, 63, 200])
def test_values_that_are_not_finite_along_a_chunk(head, before):
    """A value of a new token that is not finite makes its column NaN for the tokens from it on and
    leaves the earlier ones alone, in the first and the last of 17 tiles."""
    Tq = 1024
    pb = Problem(*head, 1, 1, Tq, [before], 64)
    clean = pb.run()
    check_some(pb, clean, [(0, 0)], "clean")
    for at in (0, 1, 64, 700, 1022, 1023):
        pg, row = int(pb.table[0, (before + at) // 64]), (before + at) % 64
        for value in (float("nan"), -float("inf")):
            old = pb.caches[2][pg, 0, row, 9].clone()
            pb.caches[2][pg, 0, row, 9] = value
            out = pb.run()
            pb.caches[2][pg, 0, row, 9] = old
            assert not torch.isfinite(out[0, 0, at:, 9]).any(), (at, value)
            out[0, 0, at:, 9] = clean[0, 0, at:, 9]
            check_some(pb, out, [(0, 0)], f"{value} at {at}")


@pytest.mark.parametrize("head", BF16)
@pytest.mark.parametrize("norm", ["rms", "group"])
def test_long_chunk_epilogue(head, norm):
    pb = Problem(*head, 2, 1, 300, [100], 16)
    g = torch.Generator().manual_seed(1)
    w, bias = (torch.randn(2, pb.Dv, generator=g) for _ in range(2))
    out = pb.run(norm=norm, norm_eps=1e-5, norm_weight=w.cuda(), norm_bias=bias.cuda(), out_scale=0.2).cpu().double()
    for b, h, o, bound in some(pb, [(0, 0), (0, 1)]):
        y, tol = ref.epilogue(o, bound, norm, 1e-5, w[h].double(), bias[h].double(), 0.2, pb.dtype)
        assert ((out[b, h] - y).abs() <= tol).all(), h


# ---------------------------------------------------------------------------
# layouts of queries and outputs
# ---------------------------------------------------------------------------
def lay_out(x, how):
    """The same queries, laid out so that the tensor cores' copies do not take them."""
    if how == "odd":                                # rows of an odd stride off 16-byte boundaries
        buf = torch.zeros(*x.shape[:3], x.shape[3] + 1, dtype=x.dtype, device="cuda")
        buf[..., 1:] = x
        return buf[..., 1:]
    if how == "rows":                               # aligned, but a row stride of 4 elements' multiple
        buf = torch.zeros(*x.shape[:3], x.shape[3] + 4, dtype=x.dtype, device="cuda")
        buf[..., :-4] = x
        return buf[..., :-4]
    assert how == "expanded"                        # one for all sequences
    return x[:1].expand(x.shape)


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,tree", [(1, False), (5, True), (17, False), (33, True), (64, True), (130, False)])
@pytest.mark.parametrize("how", ["odd", "rows", "expanded"])
def test_layouts_of_queries(head, Tq, tree, how):
    pb = Problem(*head, 4, 2, Tq, [0, 50, 300], 16, new=[Tq, max(1, Tq - 1), Tq], tree=tree)
    pb.q1, pb.q2 = lay_out(pb.q1, how), lay_out(pb.q2, how)
    check_some(pb, pb.run(), [(b, h) for b in range(3) for h in (0, 3)], f"{how} Tq={Tq}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,lens", [(1, [10, 0, 33]), (1, [3000, 5, 2]), (6, [40, 900, 1]), (20, [10, 0, 33]),
                                     (20, [3000, 5, 2]), (150, [10, 600, 33])])
@pytest.mark.parametrize("norm", [None, "rms"])
def test_misaligned_outputs(head, Tq, lens, norm):
    """Output rows that start at an odd element, of whole units and of joined ones."""
    pb = Problem(*head, 4, 2, Tq, lens, 16, new=[Tq, max(1, Tq // 2), Tq])
    buf, place = misaligned_out(pb)
    out = pb.run(out=place, norm=norm)
    assert out is place
    check_around(pb, buf, out)
    assert torch.equal(out[0], pb.run(norm=norm)[0])
    if norm is None:
        check_some(pb, out, [(b, h) for b in range(3) for h in (0, 3)], f"Tq={Tq}")
