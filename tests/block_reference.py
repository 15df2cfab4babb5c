"""The operators of a cross-attention block from their formulas, in float64 on the CPU, with
the sizes that their tests' error bounds go by."""
import torch


def head_norm(x, group, eps, w, b, scale):
    """y [B, H, T, C], and h, r, mean |x| of its rows; w, b [H, C] or None."""
    size = x.abs().mean(-1, keepdim=True)
    if group:
        x = x - x.mean(-1, keepdim=True)
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    h = x * r
    y = h if w is None else h * w[:, None]
    if b is not None:
        y = y + b[:, None]
    return scale * y, h, r, size


def head_norm_backward(x, group, eps, w, scale, dy):
    """dx, dw [H, C], db [H, C]."""
    _, h, r, _ = head_norm(x, group, eps, None, None, 1.0)
    g = scale * (dy if w is None else dy * w[:, None])
    dx = g - h * (g * h).mean(-1, keepdim=True)
    if group:
        dx = dx - g.mean(-1, keepdim=True)
    return r * dx, scale * (dy * h).sum((0, 2)), scale * dy.sum((0, 2))


U = 2.0 ** -24                  # half a float32 step, relative


class Cross:
    """Attention over an encoder's states, its gradients, and how far float32 arithmetic with
    `h` = the largest rounding of an intermediate (2^-8 in bf16, U in float32) may be off: for
    every element the sum of what each rounding puts into it, first order.

    x: q1, k1, q2, k2, v (float64 [B, heads, rows, width]); lens: states of each sequence.

    Scores: D products and sums, eS = (D + 4) U |q| |k| / sqrt(D).  Weights, relative: their own
    score's error, the largest of their row through the maximum and the sum, n + 32 roundings of
    the sum and the exponential (2^-22).  Each weight enters a product rounded by h."""

    def __init__(self, q1, k1, q2, k2, v, lam, lens, h, saved=True):
        self.x, self.lam, self.lens, self.h, self.saved = (q1, k1, q2, k2, v), lam, lens, h, saved
        B, H, Tq, D = q1.shape
        self.group = H // k1.shape[1]
        self.scale = D ** -0.5
        self.o = torch.zeros(B, H, Tq, v.shape[3], dtype=torch.float64)
        self.o_tol = torch.zeros_like(self.o)
        self.lse = torch.full((B, H, Tq, 2), -float("inf"), dtype=torch.float64)
        self.heads = {}
        for b in range(B):
            n = lens[b]
            for i in range(H):
                if n == 0:
                    continue
                hk = i // self.group
                V = v[b, hk, :n]
                A, eA, O, eO = [], [], [], []
                for q, k in ((q1, k1), (q2, k2)):
                    Q, K = q[b, i], k[b, hk, :n]
                    S = Q @ K.T * self.scale
                    eS = (D + 4) * U * (Q.abs() @ K.abs().T) * self.scale
                    A.append(torch.softmax(S, -1))
                    eA.append(eS + eS.amax(-1, keepdim=True) + (n + 32) * U)
                    O.append(A[-1] @ V)
                    eO.append((A[-1] * (h + eA[-1] + (n + 8) * U)) @ V.abs())
                    self.lse[b, i, :, len(A) - 1] = torch.logsumexp(S, -1)
                self.o[b, i] = O[0] - lam * O[1]
                self.o_tol[b, i] = eO[0] + abs(lam) * eO[1] + h * self.o[b, i].abs()
                self.heads[b, i] = (A, eA, O, eO)

    def backward(self, do):
        """{name: (gradient, bound)}, k2's beside k1's; "k" is their sum (one key tensor)."""
        q1, k1, q2, k2, v = self.x
        h, lam, scale = self.h, self.lam, self.scale
        names = ("q1", "k1", "q2", "k2", "v")
        g = {n: torch.zeros_like(t) for n, t in zip(names, self.x)}
        e = {n: torch.zeros_like(t) for n, t in zip(names, self.x)}
        dlam, elam, size = 0.0, 0.0, 0.0
        rows = do.shape[2] * self.group
        for (b, i), (A, eA, O, eO) in self.heads.items():
            n, hk = self.lens[b], i // self.group
            V, G = v[b, hk, :n], do[b, i]
            dP = G @ V.T
            edP = (V.shape[1] + 4) * U * (G.abs() @ V.abs().T)
            W = A[0] - lam * A[1]
            eW = A[0] * eA[0] + abs(lam) * A[1] * eA[1] + h * W.abs() + 4 * U * (A[0] + abs(lam) * A[1])
            g["v"][b, hk, :n] += W.T @ G
            e["v"][b, hk, :n] += (eW + rows * U * W.abs()).T @ G.abs()
            for j, c in ((0, 1.0), (1, -lam)):
                Dd = (A[j] * dP).sum(-1, keepdim=True)
                exact = (A[j] * (eA[j] * dP.abs() + edP + (n + 32) * U * dP.abs())).sum(-1, keepdim=True)
                # from the saved O and A_2 V: their errors and roundings by dO
                o2 = eO[1] + h * O[1].abs()
                from_saved = (G.abs() * (o2 if j else self.o_tol[b, i] + abs(lam) * o2)).sum(-1, keepdim=True)
                eDd = exact + (from_saved if self.saved else 0)
                dS = c * A[j] * (dP - Dd)
                edS = abs(c) * A[j] * ((eA[j] + h + 4 * U) * (dP - Dd).abs() + edP + eDd)
                Q, K = (q1, q2)[j][b, i], (k1, k2)[j][b, hk, :n]
                g[names[2 * j]][b, i] = scale * dS @ K
                e[names[2 * j]][b, i] = scale * (edS + (n + 4) * U * dS.abs()) @ K.abs()
                g[names[2 * j + 1]][b, hk, :n] += scale * dS.T @ Q
                e[names[2 * j + 1]][b, hk, :n] += scale * (edS + (rows + 4) * U * dS.abs()).T @ Q.abs()
                if j:
                    dlam -= Dd.sum()
                    elam += (exact + (from_saved if h == U else 0)).sum()
                    size += Dd.abs().sum()
        out = {n: (g[n], e[n] + h * g[n].abs()) for n in names}
        k = g["k1"] + g["k2"]
        out["k"] = (k, e["k1"] + e["k2"] + h * k.abs())
        count = do.shape[0] * do.shape[1] * do.shape[2]
        out["lam"] = (torch.as_tensor(dlam, dtype=torch.float64), torch.as_tensor(elam + (count / 128 + 64) * U * size))
        return out
