"""GPU tests of differential attention over a paged cache (new tokens and trees of
drafted tokens) against float64."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LAM = 0.8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _clean():
    da.get_device_error()
    yield
    assert da.get_device_error() == 0


class Problem:
    """Caches with the sequences' pages in a random order; unused slots and pages hold NaN."""

    def __init__(self, dtype, D, Dv, shared, H, Hk, Tq, lens, page, new=None, tree=False, seed=0, layout="head",
                 scale=1.0, slope=0.0, spikes=False):
        g = torch.Generator().manual_seed(seed + 1000 * D + Tq)
        dt = DT[dtype]
        B = len(lens)
        self.dtype, self.lens, self.new, self.Tq, self.H, self.Hk, self.Dv = dt, lens, new or [Tq] * B, Tq, H, Hk, Dv
        self.page = page
        totals = [n + t if t else 0 for n, t in zip(lens, self.new)]
        need = [-(-t // page) for t in totals]
        per = max(max(need), 1)
        pool = sum(need) + 3
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((B, per), 2 ** 30, dtype=torch.int32)       # entries past a sequence's pages are not read
        at = 0
        self.k1, self.k2, self.v = ([torch.randn(Hk, t, n, generator=g).to(dt) * s for t in totals]
                                    for n, s in ((D, scale), (D, scale), (Dv, 1.0)))
        if slope or spikes:     # scores that rise or fall along the keys, and a few that stand out
            for k in (*self.k1, *self.k2):
                along = torch.arange(k.shape[1], dtype=torch.float32)[None, :, None]
                tall = torch.where(torch.rand(Hk, k.shape[1], 1, generator=g) < 1 / 40, 6.0, 0.0) if spikes else 0.0
                k += (slope * along + tall).to(dt)
        caches = [torch.full((pool, Hk, page, n), float("nan"), dtype=dt) for n in (D, D, Dv)]
        for b, n in enumerate(need):
            ids = order[at:at + n]
            at += n
            self.table[b, :n] = ids.int()
            for cache, rows in zip(caches, (self.k1[b], self.k2[b], self.v[b])):
                full = torch.full((Hk, n * page, rows.shape[-1]), float("nan"), dtype=dt)
                full[:, :totals[b]] = rows
                cache[ids] = full.reshape(Hk, n, page, rows.shape[-1]).transpose(0, 1)
        if shared:
            self.k2 = self.k1
        self.caches = [c.cuda() for c in caches]
        if layout == "token":
            self.caches = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in self.caches]
        elif layout == "odd":
            def off(c):
                buf = torch.zeros(*c.shape[:3], c.shape[3] + 1, dtype=dt, device="cuda")
                buf[..., 1:] = c
                return buf[..., 1:]
            self.caches = [off(c) for c in self.caches]
        self.shared = shared
        self.q1, self.q2 = ((torch.randn(B, Tq, H, D, generator=g) * scale).to(dt).cuda().transpose(1, 2) for _ in range(2))
        if slope or spikes:
            self.q1, self.q2 = self.q1.abs(), self.q2.abs()
        self.tree = None
        if tree:
            back = torch.randint(1, 5, (B, Tq), generator=g)
            self.tree = torch.zeros(B, Tq, Tq, dtype=torch.bool)
            for b in range(B):
                for i in range(Tq):
                    parent = i - int(back[b, i])
                    if parent >= 0:
                        self.tree[b, i] |= self.tree[b, parent]
                    self.tree[b, i, i] = True

    def run(self, **kw):
        k1, k2, v = self.caches
        # memory that a fresh output may be given: not zeros
        torch.full((len(self.lens), self.H, self.Tq, self.Dv), float("nan"), dtype=self.dtype, device="cuda")
        args = [self.q1, k1, self.q2, k1 if self.shared else k2, v, self.table.cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda()]
        if min(self.new) < self.Tq:
            kw.setdefault("q_lengths", torch.tensor(self.new, dtype=torch.int32).cuda())
        lam = kw.pop("lam", LAM)
        if self.tree is not None:
            return da.differential_attention_tree(*args, self.tree.cuda(), lam, **kw)
        return da.differential_attention_paged(*args, lam, **kw)

    def want(self, lam=LAM):
        """[(b, h, o, bound)] of every sequence and head."""
        for b, (n, t) in enumerate(zip(self.lens, self.new)):
            if t == 0:
                continue
            tree = None if self.tree is None else self.tree[b, :t, :t]
            seen = ref.visible(n, t, tree)
            for h in range(self.H):
                hk = h // (self.H // self.Hk)
                yield b, h, *ref.attention_rows(self.q1[b, h, :t].double().cpu(), self.k1[b][hk].double(),
                                                self.q2[b, h, :t].double().cpu(), self.k2[b][hk].double(),
                                                self.v[b][hk].double(), seen, lam, self.dtype)

    def check(self, out, lam=LAM, what="", zero_rest=True):
        out = out.cpu().double()
        for b, h, o, bound in self.want(lam):
            got = out[b, h, :o.shape[0]]
            assert torch.isfinite(got).all(), f"{what} b={b} h={h}"
            over = ((got - o).abs() - bound).max()
            assert over <= 0, f"{what} b={b} h={h}: {float(over)} over the bound"
        if zero_rest:
            for b, t in enumerate(self.new):
                assert torch.count_nonzero(out[b, :, t:]) == 0


HEADS = [("bf16", 64, 128, False), ("bf16", 64, 128, True), ("bf16", 128, 128, True), ("bf16", 128, 128, False),
         ("f32", 32, 64, False), ("f32", 64, 128, True)]
# other widths run on the CUDA cores
OTHER = [("bf16", 32, 64, False), ("bf16", 128, 256, False), ("bf16", 48, 30, True), ("f32", 5, 200, False),
         ("f32", 128, 256, True), ("f32", 1, 1, False)]


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("lens", [[0], [1, 15, 16, 17], [0, 127, 128, 129, 300], [1000, 3, 0, 64, 63]])
def test_single_tokens(head, lens):
    for H, Hk, page in ((2, 2, 16), (4, 1, 64)):
        pb = Problem(*head, H, Hk, 1, lens, page, seed=len(lens))
        pb.check(pb.run(), what=f"{head} {lens}")


@pytest.mark.parametrize("head", OTHER)
@pytest.mark.parametrize("page,layout", [(16, "head"), (7, "token"), (1, "head"), (64, "odd")])
def test_other_widths_pages_and_layouts(head, page, layout):
    for Tq, new, tree in ((1, None, False), (5, [5, 2, 0], False), (9, [9, 1, 4], True)):
        pb = Problem(*head, 4, 2, Tq, [0, 33, 150], page, new=new, tree=tree, layout=layout)
        pb.check(pb.run(), what=f"{head} {page} {layout} Tq={Tq}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,H,Hk", [(2, 2, 2), (3, 6, 2), (7, 4, 4), (8, 4, 2), (16, 1, 1), (17, 2, 2), (5, 8, 1),
                                     (33, 4, 2), (64, 2, 1), (65, 2, 2), (130, 2, 1)])
@pytest.mark.parametrize("page", [16, 128])
def test_new_tokens(head, Tq, H, Hk, page):
    lens = [0, 1, 64, 200]
    new = [Tq, max(1, Tq // 2), Tq - 1, 0]
    pb = Problem(*head, H, Hk, Tq, lens, page, new=new)
    pb.check(pb.run(), what=f"{head} Tq={Tq}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,H,Hk", [(1, 2, 2), (2, 2, 1), (8, 2, 2), (15, 2, 2), (16, 4, 2), (31, 2, 1), (63, 4, 2),
                                     (64, 4, 1)])
def test_trees(head, Tq, H, Hk):
    pb = Problem(*head, H, Hk, Tq, [0, 50, 131, 64], 32, new=[Tq, Tq, max(1, Tq - 3), Tq // 2], tree=True)
    pb.check(pb.run(), what=f"{head} tree {Tq}")


@pytest.mark.parametrize("head", HEADS)
def test_many_sequences_and_idle_places(head):
    """More sequences than threads in a block, many of them idle; more units than blocks."""
    lens = [(37 * b) % 90 for b in range(600)]
    new = [b % 3 for b in range(600)]
    pb = Problem(*head, 2, 2, 2, lens, 16, new=new)
    pb.check(pb.run(), what=f"{head}")
    idle = Problem(*head, 2, 2, 2, [5, 6], 16, new=[0, 0])
    assert torch.count_nonzero(idle.run()) == 0


@pytest.mark.parametrize("head", HEADS)
def test_long_context_is_split_and_joined(head):
    """One sequence over many blocks, scores from -60 to 60 (base 2): the running maximum moves."""
    for Tq, tree in ((1, False), (4, False), (40, True)):
        pb = Problem(*head, 1, 1, Tq, [9000], 64, tree=tree, scale=2.0)
        pb.check(pb.run(), what=f"{head} {Tq}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("slope,spikes", [(0.04, False), (-0.04, False), (0.01, True), (0.0, True)])
def test_moving_maximum(head, slope, spikes):
    """Scores that pass the running maximum by more than 2^8 within a tile, between tiles and
    between the parts of a split sequence."""
    for Tq, lens in ((1, [300, 33, 1500]), (5, [100, 700]), (24, [257, 40, 600])):
        pb = Problem(*head, 2, 1, Tq, lens, 16, slope=slope if max(lens) < 1000 else slope / 3, spikes=spikes)
        pb.check(pb.run(), what=f"{head} {Tq}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [1, 20])
@pytest.mark.parametrize("at", [5, 250])
def test_visible_values_that_are_not_finite(head, Tq, at):
    """A NaN or an infinity that every row sees (inf - lambda inf) reaches its column alone."""
    pb = Problem(*head, 2, 1, Tq, [300], 16)
    clean = pb.run()
    pg, row = int(pb.table[0, at // 16]), at % 16
    for value in (float("nan"), float("inf"), -float("inf")):
        old = pb.caches[2][pg, 0, row, 7].clone()
        pb.caches[2][pg, 0, row, 7] = value
        out = pb.run()
        pb.caches[2][pg, 0, row, 7] = old
        assert torch.isnan(out[..., 7]).all(), value
        out[..., 7] = clean[..., 7]
        pb.check(out, what=f"{value}")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [3, 24])
def test_hidden_values_have_no_influence(head, Tq):
    """NaN and infinities in the keys and values of a drafted token reach only the rows that
    see it, and of the values only their own columns."""
    pb = Problem(*head, 2, 1, Tq, [37], 16, tree=True)
    clean = pb.run()
    bad = 1
    slot = pb.lens[0] + bad
    pg, row = int(pb.table[0, slot // 16]), slot % 16
    sees = pb.tree[0, :, bad]
    assert sees.any() and not sees.all()
    for value in (float("nan"), float("inf"), -float("inf")):
        old = pb.caches[2][pg, 0, row, 3].clone()
        pb.caches[2][pg, 0, row, 3] = value
        out = pb.run()
        pb.caches[2][pg, 0, row, 3] = old
        assert not torch.isfinite(out[0, :, sees][..., 3]).any()
        keep = torch.ones_like(out[0], dtype=torch.bool)
        keep[:, sees.cuda(), 3] = False
        # the other columns may take another path over the tile: to the bound
        masked = out.clone()
        masked[0][~keep] = clean[0][~keep]
        pb.check(masked, what=f"hidden value {value}")
    for cache, used in ((0, True), (1, not pb.shared)):
        old = pb.caches[cache][pg, 0, row].clone()
        pb.caches[cache][pg, 0, row] = float("nan")
        out = pb.run()
        pb.caches[cache][pg, 0, row] = old
        if used:
            assert torch.isnan(out[0, :, sees]).all()
        masked = out.clone()
        masked[:, :, sees.cuda()] = clean[:, :, sees.cuda()]
        pb.check(masked, what="hidden key")


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [4, 20])
def test_rows_that_see_nothing(head, Tq):
    pb = Problem(*head, 2, 1, Tq, [0, 20], 16, tree=True)
    pb.tree[:, 1] = False
    pb.tree[0, :, 0] = False
    pb.tree[0, 0] = False                       # sequence 0 has no cached token: rows 0 and 1 see nothing
    out = pb.run()
    assert torch.count_nonzero(out[0, :, :2]) == 0
    pb.check(out, what="empty rows")
    out = pb.run(norm="rms", norm_bias=torch.ones(2, pb.Dv, device="cuda"), out_scale=0.5)
    assert (out[0, :, :2] == 0.5).all()


@pytest.mark.parametrize("head", HEADS + OTHER[:2])
@pytest.mark.parametrize("norm", ["rms", "group", None])
@pytest.mark.parametrize("Tq,lens", [(1, [700, 5]), (3, [40]), (20, [300, 2])])
def test_epilogue(head, norm, Tq, lens):
    H = 2
    pb = Problem(*head, H, 1, Tq, lens, 16)
    g = torch.Generator().manual_seed(1)
    w, bias = (torch.randn(H, pb.Dv, generator=g) for _ in range(2))
    out = pb.run(norm=norm, norm_eps=1e-5, norm_weight=w.cuda(), norm_bias=bias.cuda(), out_scale=0.2).cpu().double()
    for b, h, o, bound in pb.want():
        y, tol = ref.epilogue(o, bound, norm, 1e-5, w[h].double(), bias[h].double(), 0.2, pb.dtype)
        assert ((out[b, h, :o.shape[0]] - y).abs() <= tol).all(), f"{head} {norm} b={b} h={h}"


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [1, 6, 30])
def test_lambda_and_cancelling_branches(head, Tq):
    pb = Problem(*head, 2, 2, Tq, [100, 3], 16)
    for lam in (-0.7, 0.0, 1.9, torch.tensor(0.6, device="cuda")):
        pb.check(pb.run(lam=lam), float(lam), f"lambda {lam}")
    pb.q2, pb.shared = pb.q1, True
    assert torch.count_nonzero(pb.run(lam=1.0)) == 0


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [2, 20])
def test_output_strides_and_rows_left_alone(head, Tq):
    pb = Problem(*head, 4, 2, Tq, [10, 0, 33], 16, new=[Tq, 0, 1])
    buf = torch.full((3, Tq, 4, pb.Dv + 8), 7.0, dtype=pb.dtype, device="cuda")
    out = buf[..., :pb.Dv].transpose(1, 2)
    assert pb.run(out=out) is out
    pb.check(out, zero_rest=False)
    assert (buf[..., pb.Dv:] == 7).all() and (out[1] == 7).all() and (out[2, :, 1:] == 7).all()


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [2, 20])
def test_out_of_range_lengths_and_pages(head, Tq):
    """A bad sequence's rows are NaN, the others are right, and the call is reported."""
    lens, page = [40, 40, 40, 40, 40], 16
    pb = Problem(*head, 2, 1, Tq, lens, page)
    good = pb.run()
    pb.check(good)
    max_keys = pb.table.shape[1] * page
    for b, change in ((1, "length"), (2, "negative"), (3, "page"), (0, "low page"), (4, "count")):
        table, ln, new = pb.table.clone(), torch.tensor(lens, dtype=torch.int32), torch.full((5,), Tq, dtype=torch.int32)
        if change == "length":
            ln[b] = max_keys - Tq + 1
        elif change == "negative":
            ln[b] = -1
        elif change == "page":
            table[b, 1] = pb.caches[0].shape[0]
        elif change == "low page":
            table[b, 0] = -1
        else:
            new[b] = Tq + 1
        k1, k2, v = pb.caches
        out = da.differential_attention_paged(pb.q1, k1, pb.q2, k1 if pb.shared else k2, v, table.cuda(), ln.cuda(), LAM,
                                              q_lengths=new.cuda())
        assert da.get_device_error() == da._lib.DIFFATTN_ERR_INDEX, change
        assert torch.isnan(out[b]).all(), change
        rest = [i for i in range(5) if i != b]
        masked = out.clone()
        masked[b] = good[b]
        pb.check(masked, what=change)
        assert torch.isfinite(out[rest]).all()


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq", [1, 20])
def test_graph_replay_follows_the_lengths(head, Tq):
    """Two calls captured into one graph each, replayed at the same time on two streams, with
    lengths that grow between replays."""
    pb = Problem(*head, 2, 1, Tq, [300, 80], 16)
    k1, k2, v = pb.caches
    table = pb.table.cuda()
    lens = torch.tensor([120, 11], dtype=torch.int32, device="cuda")
    args = (pb.q1, k1, pb.q2, k1 if pb.shared else k2, v, table, lens, LAM)
    da.differential_attention_paged(*args)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(da.differential_attention_paged(*args))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for new in ([120, 11], [300, 80], [0, 50]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        want = da.differential_attention_paged(*args)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want), new


def test_captured_with_forks_and_copies():
    """A step captured between other streams' work, copies and fills: kernels that may start
    early wait for what comes before them, whatever it is."""
    g = torch.Generator().manual_seed(21)
    B, H, Hk, D, page, n = 3, 4, 2, 64, 16, 40
    cos, sin = da.rotary_tables(128, D, device="cuda")
    table = torch.randperm(B * 4, generator=g).reshape(B, 4).int().cuda()
    k_pages, v_pages = (torch.zeros(B * 4, Hk, page, w, dtype=torch.bfloat16, device="cuda") for w in (D, 2 * D))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    q_src, k_src, v_src = (torch.zeros(B, h, n, w, dtype=torch.bfloat16, device="cuda") for h, w in ((H, D), (Hk, D), (Hk, 2 * D)))
    q, k, v = (torch.zeros_like(t) for t in (q_src, k_src, v_src))
    out = torch.zeros(B, H, n, 2 * D, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            k.copy_(k_src)
            v.copy_(v_src)
        q.copy_(q_src)
        lens.zero_()
        a, _, b, _ = da.qk_norm_rotary(q, None, q * 2, None, cos, sin)
        main.wait_stream(side)
        da.paged_cache_append(k, None, v, k_pages, None, v_pages, table, lens, None, cos, sin, norm="rms")
        o = da.differential_attention_paged(a, k_pages, b, None, v_pages, table, lens, 0.5)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            out.copy_(o)
        tree = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        t = da.differential_attention_tree(a, k_pages, b, None, v_pages, table, lens, tree, 0.5)
        main.wait_stream(side)
        return t

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tree_out = step()
    for i in range(3):
        for t in (q_src, k_src, v_src):
            t.copy_(torch.randn(t.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got, got_tree = out.clone(), tree_out.clone()
        r = da.qk_norm_rotary(q_src, k_src, q_src * 2, k_src, cos, sin)
        want = da.differential_attention(*r, v_src, 0.5)
        # both within their roundings of the exact result: weights' and outputs' of the dense one
        assert (got.float() - want.float()).abs().max() <= 4 * 2.0 ** -8 * 6
        assert torch.equal(got, got_tree)


def test_results_do_not_depend_on_the_run():
    pb = Problem("bf16", 64, 128, False, 4, 2, 6, [3000, 10, 700], 16)
    a = pb.run()
    for _ in range(3):
        assert torch.equal(a, pb.run())


def test_decode_step_as_used():
    """Prompt, append, rotate and attend, token by token and then as a drafted chain, against
    the dense forward on the rotated rows."""
    g = torch.Generator().manual_seed(3)
    B, H, Hk, T, D, page = 2, 4, 2, 70, 64, 16
    q1, q2 = (torch.randn(B, T, H, D, generator=g).to(torch.bfloat16).cuda().transpose(1, 2) for _ in range(2))
    k1, k2 = (torch.randn(B, T, Hk, D, generator=g).to(torch.bfloat16).cuda().transpose(1, 2) for _ in range(2))
    v = torch.randn(B, T, Hk, 2 * D, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
    cos, sin = da.rotary_tables(128, D, device="cuda")
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    r = da.qk_norm_rotary(q1, k1, q2, k2, cos, sin, q_weight=w, k_weight=w)
    want = da.differential_attention(*r, v, 0.6)
    table = torch.randperm(2 * B * 5, generator=g)[:B * 5].reshape(B, 5).int().cuda()
    caches = [torch.full((2 * B * 5, Hk, page, n), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (D, D, 2 * D)]
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    at = 0
    for step in (50, 1, 1, 8, 10):
        new = slice(at, at + step)
        pos = (lens[:, None] + torch.arange(step, device="cuda")[None]).int()
        a, _, b, _ = da.qk_norm_rotary(q1[:, :, new], None, q2[:, :, new], None, cos, sin, pos, q_weight=w)
        da.paged_cache_append(k1[:, :, new], k2[:, :, new], v[:, :, new], *caches, table, lens, None, cos, sin,
                              norm="rms", k_weight=w)
        if step == 8:       # the same chain as a tree
            chain = torch.ones(step, step, dtype=torch.bool, device="cuda").tril()
            o = da.differential_attention_tree(a, caches[0], b, caches[1], caches[2], table, lens, chain, 0.6)
        else:
            o = da.differential_attention_paged(a, caches[0], b, caches[1], caches[2], table, lens, 0.6)
        # the dense one rounds its weights to bf16 once, both their outputs: 2^-8 of |A| |V|
        # (at most 1.6 max|v| = 8) and twice of the output
        assert ((o.float() - want[:, :, new].float()).abs() <= 4 * 2.0 ** -8 * 8).all()
        assert (o.float() - want[:, :, new].float()).abs().mean() <= 2.0 ** -8
        lens += step
        at += step
    assert at == T


def test_more_than_2_31_elements():
    """The last pages of a cache of more than 2^31 elements."""
    g = torch.Generator().manual_seed(8)
    pages, page, Hk, D = 9000, 128, 16, 128
    kc = torch.zeros(pages, Hk, page, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(pages, Hk, page, D, dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 31
    for Tq in (1, 20):
        pb = Problem("bf16", D, D, True, Hk, Hk, Tq, [250 - Tq], page)
        table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
        for i in range(2):
            kc[pages - 1 - i] = pb.caches[0][pb.table[0, i].long()]
            vc[pages - 1 - i] = pb.caches[2][pb.table[0, i].long()]
        pb.caches, pb.table = [kc, kc, vc], table
        pb.check(pb.run(), what=f"Tq={Tq}")


def test_inference_mode():
    """A decode step in inference mode; a cache made there is not written outside of it."""
    pb = Problem("bf16", 64, 128, False, 4, 2, 3, [10, 20], 16)
    want = pb.run()
    k, v = pb.k1[0][None, :, :1].cuda().expand(2, 2, 1, 64), pb.v[0][None, :, :1].cuda().expand(2, 2, 1, 128)
    n = torch.tensor(pb.lens, dtype=torch.int32).cuda()
    with torch.inference_mode():
        made = [c.clone() for c in pb.caches]
        da.paged_cache_append(k, k.clone(), v, *made, pb.table.cuda(), n - 1)
        assert not torch.equal(made[2].nan_to_num(), pb.caches[2].nan_to_num())
        assert torch.equal(pb.run(), want)
    before = [c.clone() for c in made]
    with torch.no_grad(), pytest.raises(RuntimeError, match="inference"):
        da.paged_cache_append(k, k.clone(), v, *made, pb.table.cuda(), n)
    for a, b in zip(made, before):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())


def test_strides_of_single_heads_and_pages():
    """Dimensions of one element may have any stride: the tensor cores' copies never step them."""
    for Tq in (1, 20):
        pb = Problem("bf16", 64, 128, False, 1, 1, Tq, [30 - Tq], 32)
        want = pb.run()
        pb.check(want)
        page = [int(pb.table[0, 0])] * 3
        pb.caches = [c[p:p + 1].as_strided((1, 1, *c.shape[2:]), (0, 1, c.stride(2), 1), c[p].storage_offset())
                     for c, p in zip(pb.caches, page)]
        pb.table = torch.zeros(1, 1, dtype=torch.int32)
        q = [x.as_strided(x.shape, (3, 0, x.stride(2), 1)) for x in (pb.q1, pb.q2)]
        pb.q1, pb.q2 = q
        assert torch.equal(pb.run(), want)


def test_refusals():
    pb = Problem("bf16", 64, 128, False, 4, 2, 3, [10, 20], 16)
    k1, k2, v = pb.caches
    t, n = pb.table.cuda(), torch.tensor(pb.lens, dtype=torch.int32).cuda()
    ok = [pb.q1, k1, pb.q2, k2, v, t, n]

    def call(i=None, x=None, lam=0.5, **kw):
        a = list(ok)
        if i is not None:
            a[i] = x
        return da.differential_attention_paged(*a, lam, **kw)

    call()
    for i, x in ((0, pb.q1.float()), (0, pb.q1[0]), (2, pb.q2[:, :3]), (0, pb.q1[:, :3]), (1, k1.float()), (1, k1[:, :1]),
                 (3, k2[..., :32]), (4, v[:4]), (5, t.long()), (5, t[:1]), (6, n.long()), (6, n[:1]), (6, None),
                 (6, n.cpu()), (1, k1.transpose(2, 3).contiguous().transpose(2, 3)), (0, pb.q1.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(i, x)
    for kw in (dict(q_lengths=n.long()), dict(out=torch.empty(1, device="cuda")), dict(norm="layer"),
               dict(lam=torch.zeros(2, device="cuda")), dict(norm_weight=torch.ones(3, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(da.DiffattnError):
        call(lam=float("nan"))
    with pytest.raises(ValueError, match="forward only"):
        call(0, pb.q1.detach().requires_grad_())
    mask = torch.ones(2, 3, 3, dtype=torch.bool, device="cuda")
    da.differential_attention_tree(*ok, mask, 0.5)
    for m in (mask.int(), mask[:1], mask[..., :2], mask.cpu()):
        with pytest.raises((ValueError, TypeError)):
            da.differential_attention_tree(*ok, m, 0.5)
    big = torch.zeros(2, 4, 65, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="64"):
        da.differential_attention_tree(big, k1, big, k2, v, t, n, torch.ones(65, 65, dtype=torch.bool, device="cuda"), 0.5)
    with pytest.raises(ValueError, match="1024"):
        da.differential_attention_paged(*(x.expand(2, 4, 1025, 64) for x in (big[:, :, :1],)), k1,
                                        big[:, :, :1].expand(2, 4, 1025, 64), k2, v, t, n, 0.5)
