"""64-bit references of the serving operators: prompts of the gated delta rule,
verification of drafted trees, rows of states moved."""
import math

import torch

U = 2.0 ** -24


def gdn_prefill(q, k, v, alpha, beta, h0=None, lens=None):
    """Token after token: o [T,B,H,d] and h; alpha [T,B,H] or [T,B,H,d]."""
    T, B, H, d = q.shape
    q, k, v, beta, al = q.double(), k.double(), v.double(), beta.double(), alpha.double()
    al = al if al.dim() == 4 else al[..., None]
    h = torch.zeros(B, H, d, d, dtype=torch.float64, device=q.device) if h0 is None else h0.double().clone()
    o = torch.zeros_like(q)
    for t in range(T):
        on = torch.ones(B, dtype=torch.bool, device=q.device) if lens is None else lens.to(q.device) > t
        if not on.any():
            break
        x = h[on] * al[t, on][..., None]
        u = beta[t, on][..., None] * (v[t, on] - (x * k[t, on][..., None]).sum(-2))
        h[on] = x + k[t, on][..., None] * u[..., None, :]
        o[t, on] = (h[on] * q[t, on][..., None]).sum(-2)
    return o, h


def gdn_tolerance(d):
    """What fp32 sums may lose, as a part of the largest value.  A running sum of n terms of
    random signs is off by U sqrt(n / 6) of itself (its i-th partial sum, sqrt(i) terms large, is
    rounded with variance U^2 / 3); n = d + 64 (channels, and the tokens of a chunk).  A value of the
    state goes through three sums (what the state holds of a key, the solution among a chunk's
    tokens, the update), and the largest of 10^6 values is 6 of its standard deviations off:
    3 * 6 / sqrt(6) = 7.3, counted as 8."""
    return 8 * U * math.sqrt(d + 64)


def verify(parent, token, target, u, limit, target0=None, draft=None, draft0=None, replace=True):
    """One row by the recursion on normalised distributions.  parent, token: lists of N; target
    [N,V], draft [N,V] or None, target0, draft0 [V] or None, u: list of N + 1.  Returns the path,
    the next token, and how close the nearest decision was (a relative distance)."""
    N, V = len(parent), target.shape[1]
    d = lambda x: None if x is None else torch.nan_to_num(x.double(), nan=0.0)
    after = lambda x, x0, cur: d(x0) if cur < 0 else (None if x is None else d(x[cur]))
    path, cur, close = [], -1, 1.0
    p, q = after(target, target0, cur), after(draft, draft0, cur) if draft is not None else None
    full = p
    while len(path) < limit:
        taken = None
        for n in range(N):
            t = token[n]
            if parent[n] != cur or n <= cur or not 0 <= t < V:
                continue
            if p is None:
                taken = n
                break
            pt, lim = float(p[t]), u[n] * (1.0 if q is None else float(q[t]))
            if max(pt, lim) > 0 and pt > 0:
                close = min(close, abs(pt - lim) / max(pt, lim))
            if lim < pt:
                taken = n
                break
            if q is None:
                p = p.clone()
                p[t] = 0.0
                rest = 1.0 - pt
            else:
                p = (p - q).clamp_min(0.0)
                rest = float(p.sum())
            if not rest > 0:
                p = full
                break
            p = p / rest
            if q is not None and not replace:
                z = 1.0 - float(q[t])
                q = q.clone()
                q[t] = 0.0
                if not z > 0:
                    break
                q = q / z
        if taken is None:
            break
        path.append(taken)
        cur = taken
        p, q = after(target, target0, cur), after(draft, draft0, cur) if draft is not None else None
        full = p
    if p is None:
        return path, -1, close
    p = p.clamp_min(0.0)
    cum = p.cumsum(0)
    if not float(cum[-1]) > 0:
        return path, -1, close
    theta = u[N] * float(cum[-1])
    i = int((cum <= theta).sum())
    nxt = min(i, int((p > 0).nonzero()[-1]))
    close = min(close, float((cum - theta).abs().min()) / float(cum[-1]))
    return path, nxt, close


def gather(dst, src, index, pos, C):
    """dst, src: dicts of host arrays [rows,H,...]; returns what dst holds afterwards."""
    out = {f: x.clone() for f, x in dst.items()}
    rows = src["sq"].shape[0]
    for b, i in enumerate(index):
        for f in out:
            if f.startswith("comp") and C == 0:
                continue
            if 0 <= i < rows:
                if f.startswith("buf"):
                    if pos is not None:
                        n = max(0, min(pos[i], src[f].shape[2]))
                        out[f][b, :, :n] = src[f][i, :, :n]
                else:
                    out[f][b] = src[f][i]
            elif i == -2 and not f.startswith("buf"):
                out[f][b] = 1 if f == "col_scale" else 0
                if f == "comp_idx":
                    out[f][b] = torch.arange(C, dtype=torch.int32)
    return out
