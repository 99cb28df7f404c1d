"""64-bit references of the linear-attention operators, with their own error bounds.

Each reference returns values and, for every value, a bound on what fp32
arithmetic may lose: a sum of terms x_i formed with at most c roundings per term
is off by at most c * 2^-24 * sum |x_i| (first order), and where a sum uses an
earlier result, that result's own bound is carried through its coefficient.  The
bounds are computed from the formulas here, before any kernel output is seen.

Roundings per term, c(d) = 2 d + 64: a dot product over d channels inside a
product over d channels (2 d), and 64 for the sums over a window, a tree or a
16- or 64-token chunk (counted as blocked sums), the exponentials (an argument
|g| <= 16 that matters, off by 2^-24 |g|, and the function's own 2 ulp), the
scales and the splits of an operand into bf16 or int8 parts (2^-23 of it).
"""
import math

import torch

U = 2.0 ** -24
LOG_FORGET = -110.0      # the log decay that stands for alpha = 0


def c_of(d):
    return (2 * d + 64) * U


def half_step(dtype):
    """A rounding to dtype is off by at most this much of the value."""
    return torch.finfo(dtype).eps / 2


def log_decay(alpha):
    return torch.where(alpha == 0, torch.full_like(alpha, LOG_FORGET), alpha.log())


def la_prefill(q, k, v, alpha, h0=None, lens=None):
    """Token after token: o [T,B,H,d], h, and the same sums over absolute values."""
    T, B, H, d = q.shape
    q, k, v = q.double(), k.double(), v.double()
    al = alpha.double().expand(T, B, H)
    h = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if h0 is None else h0.double().clone()
    ha = h.abs()
    o, oa = torch.zeros_like(q), torch.zeros_like(q)
    for t in range(T):
        on = torch.ones(B, dtype=torch.bool, device=q.device) if lens is None else lens.to(q.device) > t
        if not on.any():
            break
        a = al[t, on][..., None, None]
        h[on] = a * h[on] + k[t, on][..., None] * v[t, on][..., None, :]
        ha[on] = a * ha[on] + k[t, on].abs()[..., None] * v[t, on].abs()[..., None, :]
        o[t, on] = (h[on] * q[t, on][..., None]).sum(-2)
        oa[t, on] = (ha[on] * q[t, on].abs()[..., None]).sum(-2)
    return o, h, oa, ha


def dequantize(sq_rows, r, s, idx, cv):
    """The codec's state in 64 bits; sq_rows int8 [B,H,d,d] row-major."""
    h = sq_rows.double() * r.double()[..., None] * s.double()[..., None, :]
    C = idx.shape[-1]
    if C:
        h = h.scatter_add(2, idx.long()[..., None].expand(-1, -1, -1, h.shape[-1]), cv.double())
    return h


def tree(hb, buf_k, buf_m, buf_g, pos, parent, q, k, v, alpha, beta=None, log=None):
    """The context form, node after node.  parent [B][N] as given (any values); returns o, m, g, the
    bounds of o and m, and here [B,N].  Rows with pos outside [0, W] have no nodes.  log: of alpha."""
    N, B, H, d = q.shape
    W = buf_k.shape[2]
    q, k, v = q.double(), k.double(), v.double()
    bk, bm, bg = buf_k.double(), buf_m.double(), buf_g.double()
    gd = bg.shape[-1]
    la = (log or log_decay)(alpha.double())
    la = la.expand(N, B, H)[..., None] if la.dim() < 4 else la
    c = c_of(d)
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)
    o, m, g = z(N, B, H, d), z(B, H, N, d), z(B, H, N, gd)
    eo, em = z(N, B, H, d), z(B, H, N, d)
    here = torch.zeros(B, N, dtype=torch.bool)
    for b in range(B):
        p0 = int(pos[b])
        if p0 < 0 or p0 > W:
            continue
        anc = []
        for n in range(N):
            p = int(parent[b][n])
            if p != -1 and not (0 <= p < n and here[b, p]):
                anc.append(None)
                continue
            here[b, n] = True
            anc.append([] if p == -1 else anc[p] + [p])
            gp = g[b, :, p] if p >= 0 else (bg[b, :, p0 - 1] if p0 else z(H, gd))
            gn = gp + la[n, b]
            g[b, :, n] = gn
            qn, kn = q[n, b], k[n, b]                                     # [H,d]
            ctx = [(bk[b, :, i], bm[b, :, i], bg[b, :, i], None) for i in range(p0)]
            ctx += [(k[i, b], m[b, :, i], g[b, :, i], em[b, :, i]) for i in anc[n]]
            e = gn.exp()
            vecs = [qn] if beta is None else [qn, kn]
            sums, bounds = [], []
            for x in vecs:
                y = (hb[b] * (e * x)[..., None]).sum(1)
                ya = (hb[b].abs() * (e * x).abs()[..., None]).sum(1) * c
                for kc, mc, gc, ec in ctx:
                    w = (gn - gc).exp()
                    rr = (x * w * kc).sum(-1, keepdim=True)
                    y = y + rr * mc
                    ya = ya + (x.abs() * w * kc.abs()).sum(-1, keepdim=True) * mc.abs() * c
                    if ec is not None:
                        ya = ya + rr.abs() * ec
                sums.append(y)
                bounds.append(ya)
            if beta is None:
                mn, en = v[n, b], torch.zeros_like(v[n, b])
            else:
                bt = beta[n, b].double()[:, None]
                mn = bt * (v[n, b] - sums[1])
                en = bt * (bounds[1] + 4 * U * (v[n, b].abs() + sums[1].abs()))
            m[b, :, n], em[b, :, n] = mn, en
            qk = (qn * kn).sum(-1, keepdim=True)
            o[n, b] = sums[0] + qk * mn
            eo[n, b] = bounds[0] + c * (qn * kn).abs().sum(-1, keepdim=True) * mn.abs() + qk.abs() * en
    return o, m, g, eo, em, here
