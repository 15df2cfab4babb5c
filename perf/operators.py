"""Measured cases of the operators around a paged key/value cache.

Five kinds of pass, the steps that a Differential Transformer layer makes
between its projections and its output, in training and in serving:

  rotary       per-head RMS norm and position rotation of Q1, K1, Q2, K2
  rotary_grad  the same with its backward pass (a training step's share)
  append       new keys (normed and rotated) and values into a paged cache
  paged        differential attention of new tokens over a paged cache
  tree         the same for a tree of drafted tokens

Each is computed either in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, by the calls that a
user makes of differential_attention_fwd_gb300.  exact() gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
LAMBDA = 0.8
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rotary(name, **kw):
    return dict(dict(name=name, kind="rotary", dtype="bf16", B=1, T=1, H=16, Hk=16, D=64, R=64, shared=False,
                     weights="shared", interleaved=False, start=0), **kw)


def _append(name, **kw):
    return dict(dict(name=name, kind="append", dtype="bf16", B=1, T=1, H=16, Hk=16, D=64, Dv=128, R=64, shared=False,
                     page=64, length=1024, ragged=True, norm=True, interleaved=False), **kw)


def _paged(name, **kw):
    return dict(dict(name=name, kind="paged", dtype="bf16", B=1, T=1, H=16, Hk=16, D=64, Dv=128, shared=False, page=64,
                     length=1024, ragged=True, norm=False), **kw)


def listed():
    return [
        # one decode step of 16 sequences: a few KB a head, where latency counts
        _rotary("rotary_decode_b16", B=16, start=5000),
        # the headline forward's Q and K (B2 H16 T8192 D64), a prefill
        _rotary("rotary_prefill_b2t8192", B=2, T=8192),
        # a training step of the DIFF V2 head: one key tensor, 16 over 8 heads, an odd length, a weight a head
        _rotary("rotary_train_v2_t4099", kind="rotary_grad", B=2, T=4099, Hk=8, D=128, R=128, shared=True,
                weights="per_head"),
        # a small float32 model with a part of each head rotated, in interleaved pairs
        _rotary("rotary_train_f32", kind="rotary_grad", dtype="f32", B=3, T=517, H=6, Hk=3, R=32, interleaved=True),
        # one new token for each of 16 sequences
        _append("append_token_b16", B=16, length=4000),
        # a chunk of a prefill of four sequences, ragged, DIFF V2 head
        _append("append_chunk_v2", B=4, T=2047, Hk=8, D=128, R=128, shared=True, page=128, length=3000),
        # one sequence of moderate length: the smallest call
        _paged("paged_b1_k517", length=517),
        # the decode workload of 16 sequences with 8192 keys, from pages, ragged
        _paged("paged_b16_k8192", B=16, length=8192, norm=True),
        # the DIFF V2 head over long contexts
        _paged("paged_v2_b4_k65536", B=4, Hk=8, D=128, shared=True, page=128, length=65536),
        # a small float32 model's decode step, several new tokens
        _paged("paged_f32_b4", dtype="f32", B=4, T=3, H=8, Hk=4, D=32, Dv=64, page=16, length=2900),
        # a small tree of drafted tokens for one sequence
        _paged("tree_b1_n8", kind="tree", T=8, length=1000),
        # trees of up to 61 drafted tokens for 16 sequences, DIFF V2 head
        _paged("tree_v2_b16_n61", kind="tree", B=16, T=61, Hk=8, D=128, shared=True, length=8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# The most work of a drawn case, below the largest listed one's of its kind.
_MOST_BYTES = {"rotary": 250e6, "rotary_grad": 300e6, "append": 55e6, "paged": 0.7e9, "tree": 0.35e9}
_MOST_FLOPS = {"paged": 6e10, "tree": 6e10}


def draw(rng):
    kind = rng.choice(["rotary", "rotary_grad", "append", "paged", "paged", "tree", "tree"])
    while True:
        head = rng.choice(["v1", "v1", "v2", "v2", "keys", "plain", "f32"])
        group = rng.choice([1, 1, 2, 4])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        c = dict(kind=kind, dtype="bf16", H=Hk * group, Hk=Hk, D=64, Dv=128, shared=False)
        if head == "v2":                       # the DIFF V2 head
            c.update(D=128, shared=True)
        elif head == "keys":                   # one key tensor, V = 2D
            c.update(shared=True)
        elif head == "plain":                  # two key tensors, V = D
            c.update(D=128)
        elif head == "f32":
            c.update(dtype="f32", D=rng.choice([32, 64]))
            c.update(Dv=2 * c["D"])
        if kind in ("rotary", "rotary_grad"):
            c.update(B=_log_int(rng, 1, 16), T=_log_int(rng, 1, 9000), R=rng.choice([c["D"], c["D"], c["D"] // 2]),
                     weights=rng.choice(["shared", "per_head", "none"]), interleaved=rng.random() < 0.3,
                     start=_log_int(rng, 1, 100000))
            del c["Dv"]
        else:
            c.update(B=_log_int(rng, 1, 32), length=_log_int(rng, 1, 65536), page=rng.choice([16, 32, 64, 128]),
                     ragged=rng.random() < 0.8, norm=rng.random() < 0.5)
            if kind == "append":
                c.update(T=rng.choice([1, _log_int(rng, 1, 2048)]), R=c["D"], interleaved=rng.random() < 0.3,
                         length=min(c["length"], 8192))
            elif kind == "paged":              # single tokens, a few, a chunk of a prefill
                c.update(T=rng.choice([1, 1, 1, rng.randint(2, 8), 8 if head == "f32" else _log_int(rng, 9, 300)]))
            else:
                c.update(T=rng.randint(2, 16 if head == "f32" else 64))
        w = work(c)
        if w["bytes"] <= _MOST_BYTES[kind] and w["flops"] <= _MOST_FLOPS.get(kind, 1e15):
            return c


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    keys = 1 if c["shared"] else 2
    tokens = c["B"] * c["T"]
    if c["kind"] in ("rotary", "rotary_grad"):
        values = tokens * c["D"] * (2 * c["H"] + keys * c["Hk"])
        tables = tokens * (c["R"] * 4 + 8)
        sides = 2 if c["kind"] == "rotary" else 4      # x and y; x, y, dy and dx
        return {"bytes": sides * values * size + tables, "flops": values * (10 if sides == 2 else 28)}
    if c["kind"] == "append":
        tokens = sum(_new(c))
        values = tokens * c["Hk"] * (keys * c["D"] + c["Dv"])
        return {"bytes": 2 * values * size + tokens * (c["R"] * 4 + 4), "flops": tokens * c["Hk"] * keys * c["D"] * 10}
    lens, new = _lengths(c), _new(c)
    cached = sum(n + t for n, t in zip(lens, new)) * c["Hk"] * (keys * c["D"] + c["Dv"])
    rows = sum(new) * c["H"] * (2 * c["D"] + c["Dv"])
    pairs = sum(t * n + t * (t + 1) // 2 for n, t in zip(lens, new)) * c["H"]
    return {"bytes": (cached + rows) * size, "flops": pairs * 4 * (c["D"] + c["Dv"])}


def _lengths(c):
    """Tokens cached before the call, by sequence: `length` at most, spread over
    its upper three quarters where ragged."""
    n, B = c["length"], c["B"]
    if not c["ragged"]:
        return [n] * B
    return [max(1, n - (3 * n // 4) * ((7 * b + 3) % (B + 1)) // (B + 1)) for b in range(B)]


def _new(c):
    """New tokens, by sequence: T at most."""
    T, B = c["T"], c["B"]
    if not c["ragged"] or T == 1:
        return [T] * B
    return [max(1, T - (T // 2) * ((5 * b) % B) // B) for b in range(B)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEVICE)
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device=DEVICE, dtype=torch.float32).to(dtype)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device=DEVICE)


def _tables(rows, R):
    """cos and sin of position * 10000^(-2i/R), angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=DEVICE, dtype=torch.float64) / R)
    a = torch.arange(rows, device=DEVICE, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def prepare(c, seed):
    r = _Rand(seed)
    dt = DTYPES[c["dtype"]]
    B, T, H, Hk, D = c["B"], c["T"], c["H"], c["Hk"], c["D"]
    s = dict(c)

    def heads(n, width):                       # as a projection leaves it: [B, T, heads, width], seen as [B, heads, T, width]
        return r.normal(B, T, n, width, dtype=dt).transpose(1, 2)

    if c["kind"] in ("rotary", "rotary_grad"):
        s["q1"], s["q2"], s["k1"] = heads(H, D), heads(H, D), heads(Hk, D)
        s["k2"] = s["k1"] if c["shared"] else heads(Hk, D)
        s["cos"], s["sin"] = _tables(c["start"] + T + 8 * B, c["R"])
        s["positions"] = (c["start"] + 7 * torch.arange(B, device=DEVICE)[:, None]
                          + torch.arange(T, device=DEVICE)[None, :])
        s["qw"] = s["kw"] = None
        if c["weights"] != "none":
            per = c["weights"] == "per_head"
            s["qw"] = 1 + 0.2 * r.normal(*((H, D) if per else (D,)))
            s["kw"] = 1 + 0.2 * r.normal(*((Hk, D) if per else (D,)))
        if c["kind"] == "rotary_grad":
            x = ["q1", "k1", "q2"] + ([] if c["shared"] else ["k2"])
            s["leaves"] = [s[n].requires_grad_() for n in x] + [w.requires_grad_() for w in (s["qw"], s["kw"]) if w is not None]
            s["grads"] = [r.normal(*s[n].shape, dtype=dt) for n in x]
        return s

    lens, new, page = _lengths(c), _new(c), c["page"]
    pages = [-(-(n + t) // page) for n, t in zip(lens, new)]
    per_seq = max(pages)
    pool = sum(pages) + 3
    order = r.perm(pool).to(torch.int32)
    table = torch.zeros(B, per_seq, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["lengths"] = table, _ints(lens)
    s["new"] = _ints(new) if min(new) < T else None
    s["k1c"] = r.normal(pool, Hk, page, D, dtype=dt)
    s["k2c"] = s["k1c"] if c["shared"] else r.normal(pool, Hk, page, D, dtype=dt)
    s["vc"] = r.normal(pool, Hk, page, c["Dv"], dtype=dt)
    if c["kind"] == "append":
        s["k1"], s["v"] = heads(Hk, D), heads(Hk, c["Dv"])
        s["k2"] = s["k1"] if c["shared"] else heads(Hk, D)
        s["cos"], s["sin"] = _tables(per_seq * page, c["R"])
        s["kw"] = 1 + 0.2 * r.normal(D) if c["norm"] else None
        return s
    s["q1"], s["q2"] = r.normal(B, H, T, D, dtype=dt), r.normal(B, H, T, D, dtype=dt)
    s["lam"] = torch.tensor(LAMBDA, device=DEVICE)
    s["weight"] = 1 + 0.2 * r.normal(H, c["Dv"]) if c["norm"] else None
    if c["kind"] == "tree":
        s["mask"] = _trees(B, T, seed)
    return s


def _trees(B, T, seed):
    """[B, T, T]: drafted token i sees j where j is i or an ancestor of i; a token's
    parent is one of the few before it, or the last cached token."""
    g = torch.Generator()
    g.manual_seed(seed)
    back = torch.randint(1, 6, (B, T), generator=g)
    m = torch.zeros(B, T, T, dtype=torch.bool)
    rows = torch.arange(B)
    for i in range(T):
        parent = i - back[:, i]
        m[:, i] = m[rows, parent.clamp(min=0)] & (parent >= 0)[:, None]
        m[:, i, i] = True
    return m.to(DEVICE)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"rotary": _plain_rotary, "rotary_grad": _plain_rotary_grad, "append": _plain_append, "paged": _plain_attention,
            "tree": _plain_attention}[s["kind"]](s)


def _run_own(s):
    import differential_attention_fwd_gb300 as da
    if s["kind"] in ("rotary", "rotary_grad"):
        q1, k1, q2, k2 = da.qk_norm_rotary(s["q1"], s["k1"], s["q2"], s["k2"], s["cos"], s["sin"], s["positions"],
                                           norm="rms", norm_eps=EPS, q_weight=s["qw"], k_weight=s["kw"],
                                           interleaved=s["interleaved"])
        outs = [q1, k1, q2] + ([] if s["shared"] else [k2])
        if s["kind"] == "rotary":
            return outs
        return [o.detach() for o in outs] + list(torch.autograd.grad(outs, s["leaves"], s["grads"]))
    if s["kind"] == "append":
        da.paged_cache_append(s["k1"], s["k2"], s["v"], s["k1c"], s["k2c"], s["vc"], s["table"], s["lengths"],
                              new_lengths=s["new"], cos=s["cos"], sin=s["sin"], norm="rms" if s["norm"] else None,
                              norm_eps=EPS, k_weight=s["kw"], interleaved=s["interleaved"])
        return [s["k1c"], s["vc"]] + ([] if s["shared"] else [s["k2c"]])
    kw = dict(q_lengths=s["new"])
    if s["norm"]:
        kw.update(norm="rms", norm_eps=EPS, norm_weight=s["weight"], out_scale=1 - LAMBDA)
    if s["kind"] == "tree":
        return da.differential_attention_tree(s["q1"], s["k1c"], s["q2"], s["k2c"], s["vc"], s["table"], s["lengths"],
                                              s["mask"], s["lam"], **kw)
    return da.differential_attention_paged(s["q1"], s["k1c"], s["q2"], s["k2c"], s["vc"], s["table"], s["lengths"],
                                           s["lam"], **kw)


def _plain_norm_rotate(x, w, cos, sin, interleaved, norm=True):
    """x [B, H, T, D] in 32 bits; cos, sin [B, 1, T, R/2]; w [D] or [H, D]."""
    x = x.float()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        if w is not None:
            x = x * (w if w.dim() == 1 else w[None, :, None, :])
    half = cos.shape[-1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _plain_rotary(s):
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    dt = DTYPES[s["dtype"]]
    x = [("q1", "qw"), ("k1", "kw"), ("q2", "qw")] + ([] if s["shared"] else [("k2", "kw")])
    return [_plain_norm_rotate(s[n], s[w], cos, sin, s["interleaved"]).to(dt) for n, w in x]


def _plain_rotary_grad(s):
    outs = _plain_rotary(s)
    return [o.detach() for o in outs] + list(torch.autograd.grad(outs, s["leaves"], s["grads"]))


def _plain_append(s):
    dt, page, T = DTYPES[s["dtype"]], s["page"], s["T"]
    # a token past a sequence's own new ones stands for the last of them
    i = torch.arange(T, device=DEVICE)[None, :].expand(s["B"], T)
    if s["new"] is not None:
        i = torch.minimum(i, s["new"][:, None].long() - 1)
    slot = s["lengths"][:, None].long() + i                                    # [B, T]
    pages, rows = s["table"].gather(1, slot // page).long(), slot % page
    cos, sin = s["cos"][slot][:, None], s["sin"][slot][:, None]

    def rows_of(x):                            # [B, T, Hk, width]
        return x.gather(2, i[:, None, :, None].expand(-1, x.shape[1], -1, x.shape[3])).transpose(1, 2)

    names = [("k1", "k1c")] + ([] if s["shared"] else [("k2", "k2c")])
    turned = [_plain_norm_rotate(rows_of(s[k]).transpose(1, 2), s["kw"], cos, sin, s["interleaved"], s["norm"]).to(dt)
              for k, _ in names]
    s["k1c"][pages, :, rows] = turned[0].transpose(1, 2)
    if not s["shared"]:
        s["k2c"][pages, :, rows] = turned[1].transpose(1, 2)
    s["vc"][pages, :, rows] = rows_of(s["v"])
    return [s["k1c"], s["vc"]] + ([] if s["shared"] else [s["k2c"]])


def _plain_attention(s):
    B, T, H, Hk, D, Dv = s["B"], s["T"], s["H"], s["Hk"], s["D"], s["Dv"]
    L = s["table"].shape[1] * s["page"]
    table = s["table"].long()

    def cached(x):                             # [B, Hk, L, width] in 32 bits
        return x[table].transpose(1, 2).reshape(B, Hk, L, x.shape[-1]).float()

    key = torch.arange(L, device=DEVICE)[None, None, :]
    before = s["lengths"].long()[:, None, None]
    i = torch.arange(T, device=DEVICE)[None, :, None]
    if s["kind"] == "tree":
        drafted = (key - before).clamp(0, T - 1).expand(B, T, L)
        seen = (key < before) | ((key < before + T) & s["mask"].gather(2, drafted))
    else:
        seen = key <= before + i
    if s["new"] is not None:
        seen = seen & (i < s["new"][:, None, None])
    seen = seen[:, None, None]                 # [B, 1, 1, T, L]

    def weights(q, k):
        a = q.float().reshape(B, Hk, H // Hk * T, D) @ k.transpose(-1, -2) / math.sqrt(D)
        a = a.reshape(B, Hk, H // Hk, T, L).masked_fill(~seen, -math.inf)
        top = a.amax(-1, keepdim=True)
        a = torch.exp(a - torch.where(top == -math.inf, 0.0, top))
        return a / a.sum(-1, keepdim=True).clamp(min=1e-30)

    k1 = cached(s["k1c"])
    a = weights(s["q1"], k1)
    a -= s["lam"] * weights(s["q2"], k1 if s["shared"] else cached(s["k2c"]))
    o = (a.reshape(B, Hk, H // Hk * T, L) @ cached(s["vc"])).reshape(B, H, T, Dv)
    if s["norm"]:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"][:, None, :] * (1 - LAMBDA)
    return o.to(DTYPES[s["dtype"]])


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        if c["kind"] in ("rotary", "rotary_grad"):
            return _exact_rotary(s)
        if c["kind"] == "append":
            return _exact_append(s)
        return _exact_attention(s)


def _pairs(R, interleaved):
    n = torch.arange(R // 2, device=DEVICE)
    return (2 * n, 2 * n + 1) if interleaved else (n, n + R // 2)


def _turn(x, pos, s, sign):
    """Each pair (x_a, x_b) of x [H, T, D] turned by sign * its angle at pos [T]."""
    a, b = _pairs(s["R"], s["interleaved"])
    cos, sin = s["cos"][pos].double(), sign * s["sin"][pos].double()
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _exact_rotary(s):
    names = ["q1", "k1", "q2"] + ([] if s["shared"] else ["k2"])
    outs, dxs, dws = [], [], {"qw": 0, "kw": 0}
    for j, n in enumerate(names):
        x, name = s[n].double(), "qw" if n[0] == "q" else "kw"
        w = s[name]
        D = x.shape[-1]
        w = torch.ones(D, dtype=torch.float64, device=DEVICE) if w is None else w.double()
        w = w[:, None, :] if w.dim() == 2 else w
        r = (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5)
        outs.append(torch.stack([_turn(x[b] * r[b] * w, s["positions"][b], s, 1.0) for b in range(s["B"])]))
        if s["kind"] == "rotary_grad":
            g = s["grads"][j].double()
            g = torch.stack([_turn(g[b], s["positions"][b], s, -1.0) for b in range(s["B"])])
            dw = (g * x * r).sum((0, 2))       # [H, D]
            dws[name] = dws[name] + (dw if s["weights"] == "per_head" else dw.sum(0))
            g = g * w
            dxs.append(r * g - x * r.pow(3) * (g * x).sum(-1, keepdim=True) / D)
    if s["kind"] == "rotary":
        return outs
    return outs + dxs + ([] if s["weights"] == "none" else [dws["qw"], dws["kw"]])


def _exact_append(s):
    lens, new, page = _lengths(s), _new(s), s["page"]
    caches = []
    for x, cache in (("k1", "k1c"), ("v", "vc"), ("k2", "k2c")):
        if x == "k2" and s["shared"]:
            continue
        y = s[cache].double()
        for b in range(s["B"]):
            rows = s[x][b, :, :new[b]].double()
            slot = lens[b] + torch.arange(new[b], device=DEVICE)
            if x != "v":
                if s["norm"]:
                    rows = rows / (rows.pow(2).sum(-1, keepdim=True) / s["D"] + EPS).sqrt() * s["kw"].double()
                rows = _turn(rows, slot, s, 1.0)
            y[s["table"][b, slot // page].long(), :, slot % page] = rows.transpose(0, 1)
        caches.append(y)
    return caches


def _exact_attention(s):
    lens, new = _lengths(s), _new(s)
    H, Hk, T = s["H"], s["Hk"], s["T"]
    out = torch.zeros(s["B"], H, T, s["Dv"], dtype=torch.float64, device=DEVICE)
    for b in range(s["B"]):
        n, t = lens[b], new[b]
        total = n + t
        pages = s["table"][b, :-(-total // s["page"])].long()
        hidden = torch.zeros(t, total, dtype=torch.bool, device=DEVICE)
        draft = s["mask"][b, :t, :t] if s["kind"] == "tree" else torch.ones(t, t, dtype=torch.bool, device=DEVICE).tril()
        hidden[:, n:] = ~draft
        for h in range(Hk):
            def cached(x):
                return x[pages, h].reshape(-1, x.shape[-1])[:total].double()
            own_heads = slice(h * (H // Hk), (h + 1) * (H // Hk))
            o = []
            for q, k in (("q1", "k1c"), ("q2", "k2c")):
                a = s[q][b, own_heads, :t].double() @ cached(s[k]).T * s["D"] ** -0.5
                o.append(torch.softmax(a.masked_fill(hidden, -math.inf), -1) @ cached(s["vc"]))
            out[b, own_heads, :t] = o[0] - s["lam"].double() * o[1]
    if s["norm"]:
        out = out * (out.pow(2).sum(-1, keepdim=True) / s["Dv"] + EPS).rsqrt() * s["weight"].double()[:, None, :] * (1 - LAMBDA)
    return out
