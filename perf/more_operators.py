"""Measured cases of the operators of a cross-attention block.

Seven kinds of pass, what a Differential Transformer layer over an encoder's
states, or over image and video tokens, does between its projections:

  cross       differential attention of Tq queries over an encoder's Tk states
              (padded to one length, each sequence with its own), serving
  cross_grad  the same with its backward pass (a training step's share)
  norm        the norm of each head's output (RMS, or layer norm over its
              channels), weight, bias and scale
  norm_grad   the same with its backward pass
  axes        per-head RMS norm of Q1, K1, Q2, K2 and their rotation by a
              position with several axes (time, height, width)
  axes_grad   the same with its backward pass
  axes_append new keys, normed and rotated by several axes, and values into a
              paged cache

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
def _cross(name, **kw):
    return dict(dict(name=name, kind="cross", dtype="bf16", B=1, Tq=1, Tk=77, H=16, Hk=16, D=64, Dv=128, shared=False,
                     ragged=True, empty=False, norm=False), **kw)


def _norm(name, **kw):
    return dict(dict(name=name, kind="norm", dtype="bf16", B=1, T=1, H=16, Dv=128, norm="rms", weight=True, bias=False,
                     token_major=False), **kw)


def _axes(name, **kw):
    return dict(dict(name=name, kind="axes", dtype="bf16", B=1, T=1, H=16, Hk=16, D=64, sections="8,12,12", shared=False,
                     weights="shared", interleaved=False, start=0), **kw)


def listed():
    return [
        # one token of one sequence over a short prompt's states: the smallest call
        _cross("cross_token_b1_k77", ragged=False),
        # a decoder's step: one token of each of 16 sequences over up to 1500 encoder states, the head norm fused
        _cross("cross_token_b16_k1500", B=16, Tk=1500, norm=True),
        # image tokens over an encoder's states, the DIFF V2 head, odd length, one sequence without a condition
        _cross("cross_v2_b4_q4099_k1500", B=4, Tq=4099, Tk=1500, Hk=8, D=128, shared=True, empty=True),
        # a training step of an encoder-decoder: 2047 target tokens over up to 4096 source states
        _cross("cross_train_b4_q2047_k4096", kind="cross_grad", B=4, Tq=2047, Tk=4096),
        # a training step of the DIFF V2 head: image tokens over a ragged batch of prompts
        _cross("cross_train_v2_b2_q4099_k1500", kind="cross_grad", B=2, Tq=4099, Tk=1500, Hk=8, D=128, shared=True),
        # a small float32 model's training step, odd lengths, grouped heads, one sequence without a condition
        _cross("cross_train_f32_b3_q77_k129", kind="cross_grad", dtype="f32", B=3, Tq=77, Tk=129, H=6, Hk=3, D=32, Dv=64,
               empty=True),
        # a training step's layer norm of every head at the headline forward's size (B2 H16 T8192)
        _norm("norm_train_group_b2_t8192", kind="norm_grad", B=2, T=8192, norm="group", bias=True),
        # the same of a small float32 model, RMS, odd length, rows as [B, T, H, Dv]
        _norm("norm_train_rms_f32", kind="norm_grad", dtype="f32", B=3, T=517, H=6, Dv=64, token_major=True),
        # one decode step of 16 sequences
        _norm("norm_decode_b16", B=16),
        # a prefill of image tokens with time, height and width, the DIFF V2 head
        _axes("axes_v2_b2_t8192", B=2, T=8192, Hk=8, D=128, sections="16,24,24", shared=True),
        # a training step over video tokens, an odd length, a weight a head
        _axes("axes_train_b2_t4099", kind="axes_grad", B=2, T=4099, weights="per_head"),
        # one new token for each of 16 sequences of a multimodal model, into its paged cache
        _axes("axes_append_b16", kind="axes_append", B=16, start=4000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# The most work of a drawn case, below the largest listed one's of its kind.
_MOST_BYTES = {"cross": 0.4e9, "cross_grad": 0.4e9, "norm": 200e6, "norm_grad": 330e6, "axes": 200e6, "axes_grad": 300e6,
               "axes_append": 55e6}
_MOST_FLOPS = {"cross": 2.5e11, "cross_grad": 3e11}
_MOST_FLOPS_F32 = {"cross": 2e9, "cross_grad": 1e9}


def draw(rng):
    kind = rng.choice(["cross", "cross", "cross_grad", "cross_grad", "norm", "norm_grad", "axes", "axes_grad", "axes_append"])
    while True:
        head = rng.choice(["v1", "v1", "v2", "v2", "keys", "f32"])
        group = rng.choice([1, 1, 2, 4])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        c = dict(kind=kind, dtype="bf16", B=_log_int(rng, 1, 16), H=Hk * group)
        if kind in ("cross", "cross_grad"):
            c.update(Hk=Hk, D=64, Dv=128, shared=False, Tk=_log_int(rng, 1, 6000), ragged=rng.random() < 0.8,
                     empty=rng.random() < 0.3, norm=kind == "cross" and rng.random() < 0.4)
            if kind == "cross":                # single tokens, a few, many
                c.update(Tq=rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 6000)]))
            else:
                c.update(Tq=_log_int(rng, 1, 6000), Tk=_log_int(rng, 2, 6000))    # (over one state dQ and dK are zero)
            if head == "v2":                   # the DIFF V2 head
                c.update(D=128, shared=True)
            elif head == "keys":               # one key tensor, V = 2D
                c.update(shared=True)
            elif head == "f32":
                c.update(dtype="f32", D=rng.choice([32, 64]))
                c.update(Dv=2 * c["D"])
            c["empty"] = c["empty"] and c["ragged"] and c["B"] > 1
        elif kind in ("norm", "norm_grad"):
            c.update(T=_log_int(rng, 1, 9000), Dv=128, norm=rng.choice(["rms", "group"]), weight=rng.random() < 0.8,
                     bias=rng.random() < 0.5, token_major=rng.random() < 0.5)
            c["bias"] = c["bias"] and c["weight"]
            if head == "f32":
                c.update(dtype="f32", Dv=rng.choice([64, 128]))
        else:
            c.update(T=_log_int(rng, 1, 9000), Hk=Hk, D=64, shared=head in ("v2", "keys"),
                     sections=rng.choice(["8,12,12", "16,8,8", "16,16"]), interleaved=rng.random() < 0.3,
                     weights=rng.choice(["shared", "per_head", "none"]), start=_log_int(rng, 1, 30000))
            if head == "v2":
                c.update(D=128, sections=rng.choice(["16,24,24", "32,16,16", "32,32"]))
            elif head == "f32":
                c.update(dtype="f32", D=rng.choice([32, 64]))
                c.update(sections=rng.choice(["4,8", "4,4,8"] if c["D"] == 32 else ["8,12,12", "8,8", "16,16"]))
            if kind == "axes_append":
                c.update(T=rng.choice([1, _log_int(rng, 1, 2048)]), start=min(c["start"], 8000))
        w = work(c)
        f32 = c["dtype"] == "f32"
        if w["bytes"] <= _MOST_BYTES[kind] and w["flops"] <= (_MOST_FLOPS_F32 if f32 else _MOST_FLOPS).get(kind, 1e15):
            return c


def work(c):
    size = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] in ("norm", "norm_grad"):
        values = c["B"] * c["T"] * c["H"] * c["Dv"]
        affine = c["H"] * c["Dv"] * 4 * (int(c["weight"]) + int(c["bias"]))
        grad = c["kind"] == "norm_grad"        # x and y; x, dy and dx besides
        return {"bytes": (5 if grad else 2) * values * size + (2 if grad else 1) * affine, "flops": values * (26 if grad else 8)}
    keys = 1 if c["shared"] else 2
    if c["kind"] in ("cross", "cross_grad"):
        lens = _lengths(c)
        rows = c["B"] * c["Tq"] * c["H"]
        cached = sum(lens) * c["Hk"] * (keys * c["D"] + c["Dv"])
        pairs = sum(lens) * c["Tq"] * c["H"]
        if c["kind"] == "cross":
            return {"bytes": (rows * (2 * c["D"] + c["Dv"]) + cached) * size, "flops": pairs * 4 * (c["D"] + c["Dv"])}
        padded = c["B"] * c["Tk"] * c["Hk"] * (keys * c["D"] + c["Dv"])        # their gradients are whole
        return {"bytes": (rows * (4 * c["D"] + 2 * c["Dv"]) + cached + padded) * size,
                "flops": pairs * (12 * c["D"] + 8 * c["Dv"])}
    tokens = c["B"] * c["T"]
    R = 2 * sum(_sections(c))
    turned = tokens * c["D"] * keys * c["Hk"]
    if c["kind"] == "axes_append":
        values = turned + tokens * c["Hk"] * 2 * c["D"]
        return {"bytes": 2 * values * size + tokens * (R * 4 + 8 * len(_sections(c))), "flops": turned * 10}
    values = turned + tokens * c["D"] * 2 * c["H"]
    tables = tokens * (R * 4 + 8 * len(_sections(c)))
    sides = 2 if c["kind"] == "axes" else 4    # x and y; x, y, dy and dx
    return {"bytes": sides * values * size + tables, "flops": values * (10 if sides == 2 else 28)}


def _sections(c):
    """The rotated pairs of each axis, in turn."""
    return [int(n) for n in c["sections"].split(",")]


def _lengths(c):
    """States of each sequence's own: Tk at most, spread over its upper three
    quarters where ragged; the last sequence has none where `empty`."""
    n, B = c["Tk"], c["B"]
    lens = [max(1, n - (3 * n // 4) * ((7 * b + 3) % (B + 1)) // (B + 1)) for b in range(B)] if c["ragged"] else [n] * B
    if c["empty"]:
        lens[-1] = 0
    return lens


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


def _tables(rows, sections):
    """cos and sin of position * 10000^(-i / n) for the n pairs i of each axis, side
    by side; angles in 64 bits."""
    f = torch.cat([10000.0 ** (-torch.arange(n, device=DEVICE, dtype=torch.float64) / n) for n in sections])
    a = torch.arange(rows, device=DEVICE, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _grid(c):
    """Positions [B, T, axes] of image or video tokens in raster order, from `start`:
    the frame, then the row and the column within it, as many axes as there are."""
    B, T, n = c["B"], c["T"], len(_sections(c))
    t = torch.arange(T, device=DEVICE)
    side = max(1, int(math.sqrt(min(T, 1024))))
    axes = [t // (side * side), t // side % side, t % side] if n == 3 else [t // side, t % side]
    first = c["start"] + 7 * torch.arange(B, device=DEVICE)
    return first[:, None, None] + torch.stack(axes, -1)[None]


def prepare(c, seed):
    r = _Rand(seed)
    dt = DTYPES[c["dtype"]]
    B, H = c["B"], c["H"]
    s = dict(c)

    def heads(T, n, width):                    # as a projection leaves it: [B, T, heads, width], seen as [B, heads, T, width]
        return r.normal(B, T, n, width, dtype=dt).transpose(1, 2)

    if c["kind"] in ("cross", "cross_grad"):
        D, Dv, Hk = c["D"], c["Dv"], c["Hk"]
        s["q1"], s["q2"] = heads(c["Tq"], H, D), heads(c["Tq"], H, D)
        # what the decoder's layer projected once from the encoder's states
        s["k1"] = heads(c["Tk"], Hk, D)
        s["k2"] = s["k1"] if c["shared"] else heads(c["Tk"], Hk, D)
        s["v"] = heads(c["Tk"], Hk, Dv)
        lens = _lengths(c)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE) if min(lens) < c["Tk"] else None
        s["lam"] = torch.tensor(LAMBDA, dtype=dt, device=DEVICE)      # a parameter of the model, of its type
        s["weight"] = 1 + 0.2 * r.normal(H, Dv) if c["norm"] else None
        if c["kind"] == "cross_grad":
            s["leaves"] = [s[n].requires_grad_() for n in ["q1", "k1", "q2"] + ([] if c["shared"] else ["k2"]) + ["v", "lam"]]
            s["grad"] = r.normal(B, H, c["Tq"], Dv, dtype=dt)
        return s
    if c["kind"] in ("norm", "norm_grad"):
        T, Dv = c["T"], c["Dv"]
        s["x"] = heads(T, H, Dv) if c["token_major"] else r.normal(B, H, T, Dv, dtype=dt)
        s["w"] = 1 + 0.2 * r.normal(H, Dv) if c["weight"] else None
        s["b"] = 0.2 * r.normal(H, Dv) if c["bias"] else None
        if c["kind"] == "norm_grad":
            s["leaves"] = [t.requires_grad_() for t in (s["x"], s["w"], s["b"]) if t is not None]
            s["grad"] = heads(T, H, Dv) if c["token_major"] else r.normal(B, H, T, Dv, dtype=dt)
        return s

    T, Hk, D = c["T"], c["Hk"], c["D"]
    s["positions"] = _grid(c)
    s["cos"], s["sin"] = _tables(int(c["start"] + 7 * B + T + 1), _sections(c))
    s["k1"] = heads(T, Hk, D)
    s["k2"] = s["k1"] if c["shared"] else heads(T, Hk, D)
    s["qw"] = s["kw"] = None
    if c["weights"] != "none":
        per = c["weights"] == "per_head"
        s["qw"] = 1 + 0.2 * r.normal(*((H, D) if per else (D,)))
        s["kw"] = 1 + 0.2 * r.normal(*((Hk, D) if per else (D,)))
    if c["kind"] == "axes_append":
        # pages of 64 slots, in any order; `start` tokens are cached
        s["v"] = heads(T, Hk, 2 * D)
        pages = -(-(c["start"] + T) // 64)
        s["table"] = r.perm(B * pages).to(torch.int32).reshape(B, pages)
        s["lengths"] = torch.full((B,), c["start"], dtype=torch.int32, device=DEVICE)
        # zeros stand for what earlier calls wrote
        s["k1c"] = torch.zeros(B * pages, Hk, 64, D, dtype=dt, device=DEVICE)
        s["k2c"] = s["k1c"] if c["shared"] else torch.zeros_like(s["k1c"])
        s["vc"] = torch.zeros(B * pages, Hk, 64, 2 * D, dtype=dt, device=DEVICE)
        return s
    s["q1"], s["q2"] = heads(T, H, D), heads(T, H, D)
    if c["kind"] == "axes_grad":
        x = ["q1", "k1", "q2"] + ([] if c["shared"] else ["k2"])
        s["leaves"] = [s[n].requires_grad_() for n in x] + [w.requires_grad_() for w in (s["qw"], s["kw"]) if w is not None]
        s["grads"] = [r.normal(*s[n].shape, dtype=dt) for n in x]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    """The pass's outputs; with a gradient, the results and then the gradients."""
    kind = s["kind"].split("_")[0]
    forward = {"cross": _own_cross, "norm": _own_norm, "axes": _own_axes} if own else \
        {"cross": _plain_cross, "norm": _plain_norm, "axes": _plain_axes}
    outs = forward[kind](s)
    if not s["kind"].endswith("_grad"):
        return outs
    grads = s["grads"] if kind == "axes" else [s["grad"]]
    return [o.detach() for o in outs] + list(torch.autograd.grad(outs, s["leaves"], grads))


def _own_cross(s):
    import differential_attention_fwd_gb300 as da
    kw = dict(norm="rms", norm_eps=EPS, norm_weight=s["weight"], out_scale=1 - LAMBDA) if s["norm"] else {}
    return [da.differential_cross_attention(s["q1"], s["k1"], s["q2"], s["k2"], s["v"], s["lam"], kv_lengths=s["lens"], **kw)]


def _own_norm(s):
    import differential_attention_fwd_gb300 as da
    return [da.differential_head_norm(s["x"], norm=s["norm"], norm_eps=EPS, norm_weight=s["w"], norm_bias=s["b"],
                                      out_scale=1 - LAMBDA)]


def _own_axes(s):
    import differential_attention_fwd_gb300 as da
    sections = tuple(_sections(s))
    if s["kind"] == "axes_append":
        da.paged_cache_append(s["k1"], s["k2"], s["v"], s["k1c"], s["k2c"], s["vc"], s["table"], s["lengths"],
                              cos=s["cos"], sin=s["sin"], positions=s["positions"], sections=sections, norm="rms",
                              norm_eps=EPS, k_weight=s["kw"], interleaved=s["interleaved"])
        return [s["k1c"], s["vc"]] + ([] if s["shared"] else [s["k2c"]])
    q1, k1, q2, k2 = da.qk_norm_rotary(s["q1"], s["k1"], s["q2"], s["k2"], s["cos"], s["sin"], s["positions"],
                                       norm="rms", norm_eps=EPS, q_weight=s["qw"], k_weight=s["kw"],
                                       interleaved=s["interleaved"], sections=sections)
    return [q1, k1, q2] + ([] if s["shared"] else [k2])


def _plain_cross(s):
    B, Tq, Tk, H, Hk, D = s["B"], s["Tq"], s["Tk"], s["H"], s["Hk"], s["D"]
    hidden = None
    if s["lens"] is not None:
        hidden = (torch.arange(Tk, device=DEVICE) >= s["lens"][:, None])[:, None, None]       # [B, 1, 1, Tk]

    def weights(q, k):
        a = (q.float().reshape(B, Hk, H // Hk * Tq, D) @ k.transpose(-1, -2)) / math.sqrt(D)
        if hidden is not None:
            a = a.masked_fill(hidden, -math.inf)
        top = a.detach().amax(-1, keepdim=True)
        a = torch.exp(a - torch.where(top == -math.inf, 0.0, top))
        return a / a.sum(-1, keepdim=True).clamp(min=1e-30)

    k1, v = s["k1"].float(), s["v"].float()
    if hidden is not None:                     # what lies behind a sequence's own states is not looked at
        v = v.masked_fill(hidden.transpose(-1, -2), 0.0)
    a = weights(s["q1"], k1) - s["lam"] * weights(s["q2"], k1 if s["shared"] else s["k2"].float())
    o = (a @ v).reshape(B, H, Tq, s["Dv"])
    if s["norm"]:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"][:, None, :] * (1 - LAMBDA)
    return [o.to(DTYPES[s["dtype"]])]


def _plain_norm(s):
    x = s["x"].float()
    if s["norm"] == "group":
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    if s["w"] is not None:
        y = y * s["w"][:, None, :]
    if s["b"] is not None:
        y = y + s["b"][:, None, :]
    return [(y * (1 - LAMBDA)).to(DTYPES[s["dtype"]])]


def _plain_norm_rotate(x, w, cos, sin, interleaved):
    """x [B, heads, T, D]; cos, sin [B, 1, T, pairs]; w [D] or [heads, D]."""
    x = x.float()
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


def _plain_axes(s):
    dt, at = DTYPES[s["dtype"]], 0
    cos, sin = [], []
    for i, n in enumerate(_sections(s)):       # the columns of each axis, by its own position
        p = s["positions"][..., i]
        cos.append(s["cos"][:, at:at + n][p])
        sin.append(s["sin"][:, at:at + n][p])
        at += n
    cos, sin = torch.cat(cos, -1)[:, None], torch.cat(sin, -1)[:, None]
    x = [("k1", "kw")] + ([] if s["shared"] else [("k2", "kw")])
    if s["kind"] != "axes_append":
        x = [("q1", "qw"), ("k1", "kw"), ("q2", "qw")] + x[1:]
    outs = [_plain_norm_rotate(s[n], s[w], cos, sin, s["interleaved"]).to(dt) for n, w in x]
    if s["kind"] != "axes_append":
        return outs
    slot = s["lengths"][:, None].long() + torch.arange(s["T"], device=DEVICE)             # [B, T]
    pages, rows = s["table"].long().gather(1, slot // 64), slot % 64
    s["k1c"][pages, :, rows] = outs[0].transpose(1, 2)
    if not s["shared"]:
        s["k2c"][pages, :, rows] = outs[1].transpose(1, 2)
    s["vc"][pages, :, rows] = s["v"].transpose(1, 2)
    return [s["k1c"], s["vc"]] + ([] if s["shared"] else [s["k2c"]])


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"cross": _exact_cross, "norm": _exact_norm, "axes": _exact_axes}[c["kind"].split("_")[0]](s)


def _exact_cross(s):
    B, H, Tq, Tk, D = s["B"], s["H"], s["Tq"], s["Tk"], s["D"]
    group = H // s["Hk"]
    f8 = dict(dtype=torch.float64, device=DEVICE)
    out = torch.zeros(B, H, Tq, s["Dv"], **f8)
    grad = s["kind"] == "cross_grad"
    if grad:
        g = {n: torch.zeros(s[n].shape, **f8) for n in ("q1", "k1", "q2", "k2", "v")}
        dlam = torch.zeros((), **f8)
    lam = s["lam"].double()
    for b, n in enumerate(_lengths(s)):
        if n == 0:                             # no state: zeros, and no gradient
            continue
        for h in range(H):
            hk = h // group
            v = s["v"][b, hk, :n].double()
            q = [s[x][b, h].double() for x in ("q1", "q2")]
            k = [s[x][b, hk, :n].double() for x in ("k1", "k2")]
            A = [torch.softmax(q[i] @ k[i].T * D ** -0.5, -1) for i in (0, 1)]
            out[b, h] = A[0] @ v - lam * (A[1] @ v)
            if not grad:
                continue
            do = s["grad"][b, h].double()
            dP = do @ v.T
            g["v"][b, hk, :n] += (A[0] - lam * A[1]).T @ do
            for i, sign in ((0, 1.0), (1, -lam)):
                rows = (A[i] * dP).sum(-1, keepdim=True)
                dS = sign * A[i] * (dP - rows) * D ** -0.5
                g["q1" if i == 0 else "q2"][b, h] = dS @ k[i]
                g["k1" if i == 0 else "k2"][b, hk, :n] += dS.T @ q[i]
                if i == 1:
                    dlam -= rows.sum()
    if s["norm"]:
        out = out * (out.pow(2).sum(-1, keepdim=True) / s["Dv"] + EPS).rsqrt() * s["weight"].double()[:, None, :] * (1 - LAMBDA)
    if not grad:
        return [out]
    if s["shared"]:
        return [out, g["q1"], g["k1"] + g["k2"], g["q2"], g["v"], dlam]
    return [out, g["q1"], g["k1"], g["q2"], g["k2"], g["v"], dlam]


def _exact_norm(s):
    x = s["x"].double()
    n = s["Dv"]
    w = (torch.ones(s["H"], 1, n, dtype=torch.float64, device=DEVICE) if s["w"] is None else s["w"].double()[:, None])
    if s["norm"] == "group":
        x = x - x.sum(-1, keepdim=True) / n
    r = (x.pow(2).sum(-1, keepdim=True) / n + EPS).rsqrt()
    h = x * r
    y = h * w if s["b"] is None else h * w + s["b"].double()[:, None]
    scale = 1 - LAMBDA
    if s["kind"] == "norm":
        return [y * scale]
    dy = s["grad"].double() * scale
    g = dy * w
    dx = g - h * (g * h).sum(-1, keepdim=True) / n
    if s["norm"] == "group":
        dx = dx - g.sum(-1, keepdim=True) / n
    out = [y * scale, dx * r]
    if s["w"] is not None:
        out.append((dy * h).sum((0, 2)))
    if s["b"] is not None:
        out.append(dy.sum((0, 2)))
    return out


def _exact_axes(s):
    sections = _sections(s)
    axis = torch.tensor([i for i, n in enumerate(sections) for _ in range(n)], device=DEVICE)     # of each pair
    pair = torch.arange(len(axis), device=DEVICE)
    a, b = (2 * pair, 2 * pair + 1) if s["interleaved"] else (pair, pair + len(axis))

    def turn(x, i, sign):                      # x [heads, T, D] of sequence i
        at = s["positions"][i][:, axis]        # [T, pairs]
        cos, sin = s["cos"][at, pair].double(), sign * s["sin"][at, pair].double()
        y = x.clone()
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return y

    names = ["k1"] + ([] if s["shared"] else ["k2"])
    if s["kind"] != "axes_append":
        names = ["q1", "k1", "q2"] + names[1:]
    outs, dxs, dws = [], [], {"qw": 0, "kw": 0}
    for j, n in enumerate(names):
        x, name = s[n].double(), "qw" if n[0] == "q" else "kw"
        w = s[name]
        D = x.shape[-1]
        w = torch.ones(D, dtype=torch.float64, device=DEVICE) if w is None else w.double()
        w = w[:, None, :] if w.dim() == 2 else w
        r = (x.pow(2).sum(-1, keepdim=True) / D + EPS).pow(-0.5)
        outs.append(torch.stack([turn(x[i] * r[i] * w, i, 1.0) for i in range(s["B"])]))
        if s["kind"] == "axes_grad":
            g = s["grads"][j].double()
            g = torch.stack([turn(g[i], i, -1.0) for i in range(s["B"])])
            dw = (g * x * r).sum((0, 2))       # [heads, D]
            dws[name] = dws[name] + (dw if s["weights"] == "per_head" else dw.sum(0))
            g = g * w
            dxs.append(r * g - x * r.pow(3) * (g * x).sum(-1, keepdim=True) / D)
    if s["kind"] == "axes":
        return outs
    if s["kind"] == "axes_grad":
        return outs + dxs + ([] if s["weights"] == "none" else [dws["qw"], dws["kw"]])
    caches = []
    for rows, cache in [(outs[0], "k1c"), (s["v"].double(), "vc")] + ([] if s["shared"] else [(outs[1], "k2c")]):
        y = s[cache].double()
        for i in range(s["B"]):
            slot = s["start"] + torch.arange(s["T"], device=DEVICE)
            y[s["table"][i, slot // 64].long(), :, slot % 64] = rows[i].transpose(0, 1)
        caches.append(y)
    return caches
