"""Measured cases of the serving operators around the recurrent state.

Three operators, each in a plain form (elementary torch operations) and through
the library's entry points:

* ``prompt``  the gated delta rule over a padded batch of prompts,
              H <- (I - beta k k^T) D H + beta k v^T, o = H^T q with D = alpha I
              or diag(alpha) (``lq_gdn_prefill_ragged``); one token is its
              recurrent form over the fp32 state;
* ``verify``  drafted trees against the target's probabilities with given random
              numbers: the accepted path of every row and the token after it
              (``lq_tree_verify``);
* ``gather``  rows of the layers' quantized states and windows copied, forked,
              compacted and cleared by an index per row (``lq_state_gather``).
"""
import math
import random

import torch

own = False

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64      # tokens per chunk of the plain prompt (16 with a decay per key channel)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _prompt(name, B, H, d, T, io, per_key=False, ragged=False, start=True):
    return dict(name=name, op="prompt", B=B, H=H, d=d, T=T, io=io, per_key=per_key, ragged=ragged, start=start)


def _verify(name, B, N, depth, V, W, draft, root=False, ragged=True, cut=False):
    """draft: "none" (drafts without probabilities), "with" or "without" replacement among a node's
    children; root: the token after the window is drafted too (else it is the tree's first node);
    cut: the target keeps only tokens of at least a twentieth of its largest probability."""
    return dict(name=name, op="verify", B=B, N=N, depth=depth, V=V, W=W, draft=draft, root=root, ragged=ragged,
                cut=cut)


def _gather(name, kind, layers, B, H, d, W, C, per_key=False):
    """kind: "admit" (rows of another batch), "beams" (any row to any row, into a second set of states),
    "fork" and "compact" (in place)."""
    return dict(name=name, op="gather", kind=kind, layers=layers, B=B, H=H, d=d, W=W, C=C, per_key=per_key)


def listed():
    return [
        # one token of every sequence of a serving batch, over fp32 states
        _prompt("prompt one token", 64, 32, 128, 1, "bf16"),
        # a short prompt of one sequence: latency
        _prompt("prompt short", 1, 16, 128, 512, "bf16", start=False),
        # one long document: few heads, many tokens
        _prompt("prompt long", 1, 16, 128, 16384, "bf16", start=False),
        # a padded batch of prompts of different lengths, continued from earlier states, fp32 tokens
        _prompt("prompt padded batch", 24, 8, 128, 1021, "f32", ragged=True),
        # a full batch of prompts
        _prompt("prompt batch", 64, 32, 128, 512, "bf16", start=False),
        # a full batch with a decay per key channel
        _prompt("prompt per-key batch", 32, 32, 128, 512, "bf16", per_key=True, ragged=True),
        # a few drafted tokens of one sequence, drafted one after another: latency
        _verify("verify one sequence", 1, 8, 8, 32000, 16, "with", ragged=False),
        # chains of looked-up tokens (no draft probabilities), an odd vocabulary, a filtered target
        _verify("verify chains", 256, 5, 5, 50021, 16, "none", root=True, cut=True),
        # a serving batch with a drafted tree per sequence
        _verify("verify trees", 64, 32, 8, 131072, 16, "without"),
        # one prompt's states enter a serving batch: latency
        _gather("gather admit", "admit", 24, 64, 16, 128, 16, 4),
        # sequences fork into several samples, in place
        _gather("gather fork", "fork", 2, 64, 32, 128, 16, 4),
        # sequences end: the last rows move into their places, in place
        _gather("gather compact batch", "compact", 1, 256, 32, 128, 16, 4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for x in m:
            m[x] = max(m[x], w[x])
    op = rng.choice(["prompt", "verify", "gather"])
    while True:
        B, H = _log_int(rng, 1, 256), _log_int(rng, 1, 64)
        d = rng.choice([16, 64, 128, 128, 128])
        W, C = rng.choice([4, 8, 13, 16, 16, 32]), rng.randint(0, 8)
        per_key = rng.random() < 0.35
        ragged = rng.random() < 0.7
        if op == "prompt":
            c = _prompt("", B, H, d, _log_int(rng, 1, 16384), rng.choice(["f32", "bf16", "bf16"]), per_key, ragged,
                        rng.random() < 0.5)
        elif op == "verify":
            N = _log_int(rng, 1, 64)
            c = _verify("", B, N, rng.randint(1, min(N, 16)), _log_int(rng, 100, 131072), W,
                        rng.choice(["none", "with", "without"]), rng.random() < 0.5, ragged, rng.random() < 0.5)
        else:
            c = _gather("", rng.choice(["admit", "beams", "fork", "compact"]), rng.randint(1, 32), B, H, d, W, C, per_key)
        w = work(c)
        if op == "gather" and w["bytes"] <= 12 * B:         # nothing would move
            continue
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"] and _held(c) <= 3e9:
            del c["name"]
            return c


def _held(c):
    """Bytes of the case's inputs, about."""
    if c["op"] == "verify":
        return 8 * (c["N"] + 1) * c["B"] * c["V"]
    if c["op"] == "gather":
        return 2 * c["layers"] * c["B"] * c["H"] * (c["d"] ** 2 + 8 * c["d"] + 4 * c["C"] * (c["d"] + 1) +
                                                    c["W"] * 4 * (2 * c["d"] + (c["d"] if c["per_key"] else 1)))
    return c["T"] * c["B"] * c["H"] * c["d"] * 16


def _lens(c):
    """Tokens of each row of a prompt batch (from the whole length down to one)."""
    T, B = c["T"], c["B"]
    return [max(1, T - (b * 5 % B) * T // B) for b in range(B)] if c["ragged"] else [T] * B


def _positions(c, n=None):
    """Window positions of the rows, in [0, W]."""
    n = c["B"] if n is None else n
    return [(7 * b + 3) % (c["W"] + 1) if c.get("ragged", True) else c["W"] // 2 for b in range(n)]


def _trees(c):
    """Per row the parents of its N nodes (-1: the last committed token; -2: no node).  Chains where
    the depth is the number of nodes."""
    N = c["N"]
    rng = random.Random(1000 * N + c["depth"])
    out = []
    for b in range(c["B"]):
        if b >= 8:
            out.append(list(out[b % 8]))
            continue
        par, dep = [], []
        for n in range(N):
            p = n - 1 if c["depth"] == N or rng.random() < 0.45 else rng.randrange(n) if n else -1
            while p >= 0 and dep[p] + 1 > c["depth"]:
                p = par[p]
            if p == -1 and n and not c["root"]:
                p = 0 if c["depth"] > 1 else -2
            par.append(p)
            dep.append(0 if p == -2 else 1 if p < 0 else dep[p] + 1)
        out.append(par)
    if c["ragged"]:                                       # some rows drafted fewer tokens
        for b, par in enumerate(out):
            keep = N - (3 * b) % (N // 2 + 1)
            out[b] = par[:keep] + [-2] * (N - keep)
    return out


def _index(c):
    """The source row of every row (-1: stays, -2: cleared) and the number of source rows."""
    B, kind = c["B"], c["kind"]
    if kind == "admit":                                   # every 16th row takes one of the admitted sequences
        n = max(1, B // 16)
        return [b // 16 % n if b % 16 == 5 % min(B, 16) else -1 for b in range(B)], n
    if kind == "beams":                                   # four beams a sequence, the best ones survive
        return [min(B - 1, b // 4 * 4 + (b * b + 1) % 4) for b in range(B)], B
    if kind == "fork":                                    # eight samples of every eighth row
        return [b // 8 * 8 for b in range(B)], B
    # compact: a third of the rows ended; the last live rows move into the first holes, the rest is cleared
    live = [b for b in range(B) if b % 3 != 1]
    idx = [-1 if b in set(live) else -2 for b in range(B)]
    holes, tail = [b for b in range(len(live)) if idx[b] == -2], [b for b in live if b >= len(live)]
    for b, x in zip(holes, tail):
        idx[b] = x
    return idx, B


def work(case):
    c = case
    B = c["B"]
    if c["op"] == "prompt":
        H, d = c["H"], c["d"]
        es = 4 if c["io"] == "f32" else 2
        n = sum(_lens(c)) * H
        by = n * (4 * d * es + 4 + 4 * (d if c["per_key"] else 1)) + B * H * d * d * 4 * (2 if c["start"] else 1)
        return {"bytes": by, "flops": n * 6 * d * d}
    if c["op"] == "verify":
        # one row of the target (and of the draft) for the token after the path, and the nodes' own numbers
        rows = 1 if c["draft"] == "none" else 2
        nodes = sum(p != -2 for par in _trees(c) for p in par)
        return {"bytes": B * c["V"] * 4 * rows + nodes * (12 + 4 * rows) + B * (4 * c["depth"] + 16),
                "flops": B * c["V"] * 2 * rows}
    idx, n = _index(c)
    H, d, C = c["H"], c["d"], c["C"]
    head = d * d + 8 * d + C * (4 * d + 4)
    slot = 4 * (2 * d + (d if c["per_key"] else 1))
    pos = _positions(c, n)
    moved = [i for b, i in enumerate(idx) if i >= 0 and not (c["kind"] in ("fork", "compact") and i == b)]
    by = sum(head + slot * pos[i] for i in moved) + sum(head + slot * pos[i] for i in set(moved))
    by += head * sum(i == -2 for i in idx)
    return {"bytes": by * H * c["layers"] + 12 * B, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _byte_order(d, device):
    """off[i, j]: the place of byte (i, j) among a head's d*d stored bytes."""
    i = torch.arange(d, device=device)[:, None]
    j = torch.arange(d, device=device)[None, :]
    G, KS = min(4, d // 16), (d + 63) // 64
    return ((((j // 16) * KS + i // 64) * G + (i % 64) // 16) * 16 + j % 16) * 16 + i % 16


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


FIELDS = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")


def _states(c, B, g, dev):
    """The layers' codecs and windows of B rows, [layers,B,...]."""
    H, d, W, C = c["H"], c["d"], c["W"], c["C"]
    rn = lambda *s: torch.randn((c["layers"], *s), device=dev, generator=g)
    ru = lambda *s: torch.rand((c["layers"], *s), device=dev, generator=g)
    gd = d if c["per_key"] else 1
    idx = ru(B, H, d).topk(max(C, 1), dim=-1).indices.sort(dim=-1).values
    sq = (40 * rn(B, H, d, d)).round_().clamp_(-127, 127)
    if C:
        sq.scatter_(3, idx[..., None].expand(-1, -1, -1, -1, d), 0.0)
    flat = torch.empty((c["layers"], B, H, d * d), device=dev, dtype=torch.int8)
    flat[..., _byte_order(d, dev).reshape(-1)] = sq.to(torch.int8).reshape(flat.shape)
    gates = torch.sigmoid(3.0 - 0.5 * rn(B, H, W, gd))
    return dict(sq=flat, row_scale=(0.5 + ru(B, H, d)) / 127, col_scale=0.2 + ru(B, H, d),
                comp_idx=idx.to(torch.int32), comp_val=1.5 * rn(B, H, max(C, 1), d), buf_k=_unit(rn(B, H, W, d)),
                buf_m=0.5 * rn(B, H, W, d), buf_g=gates.log().cumsum(3))


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(s, device=dev, generator=g)
    ru = lambda *s: torch.rand(s, device=dev, generator=g)
    int32 = lambda x: torch.tensor(x, device=dev, dtype=torch.int32)
    s = dict(case=c)
    B = c["B"]
    if c["op"] == "prompt":
        T, H, d, io = c["T"], c["H"], c["d"], IO[c["io"]]
        s["q"], s["k"] = _unit(rn(T, B, H, d)).to(io), _unit(rn(T, B, H, d)).to(io)
        s["v"] = rn(T, B, H, d).to(io)
        # gates as trained ones give them: decays of about 0.95 a token, steps of any size
        s["alpha"] = torch.sigmoid(3.0 - 0.5 * rn(T, B, H, d) if c["per_key"] else 3.0 - 0.5 * rn(T, B, H))
        s["beta"] = torch.sigmoid(1.5 * rn(T, B, H))
        s["h0"] = 0.3 * rn(B, H, d, d) if c["start"] else None
        s["lens"] = int32(_lens(c)) if c["ragged"] else None
        s["h"], s["o"] = torch.zeros((B, H, d, d), device=dev), torch.zeros((T, B, H, d), device=dev, dtype=io)
        if own:
            from recurrent_state_quant_lq_amd import lq
            s["dims"] = lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_PER_KEY if c["per_key"] else lq.LQ_DECAY_SCALAR,
                                     1, lq.LQ_IO_BF16 if c["io"] == "bf16" else lq.LQ_IO_F32)
            s["work"] = torch.zeros((lq.lq_gdn_workspace_bytes(s["dims"], T),), device=dev, dtype=torch.uint8)
        return s
    if c["op"] == "verify":
        N, V = c["N"], c["V"]
        # the draft follows the target (after every node, the last row after the committed tokens)
        logits = 4.0 * rn(N + 1, B, V)
        t = torch.softmax(logits, -1)
        if c["cut"]:
            t = torch.where(t >= 0.05 * t.amax(-1, keepdim=True), t, 0.0)
            t /= t.sum(-1, keepdim=True)
        q = torch.softmax(logits + 0.7 * rn(N + 1, B, V), -1)
        trees = _trees(c)
        parent = int32(trees)
        # every node's token from the draft after its parent (looked up: from the target itself);
        # without replacement: the siblings are the largest of q / e, e one exponential variable a token
        rank = []
        for par in trees:
            rank.append([sum(x == p for x in par[:n]) for n, p in enumerate(par)])
        rows = torch.where(parent < 0, N, parent).long().T                       # [N,B]
        cols = torch.arange(B, device=dev)
        if c["draft"] == "without":
            most = min(V, 1 + max(max(r) for r in rank))
            best = (q / -torch.log1p(-ru(N + 1, B, V)).clamp_min(1e-30)).topk(most, dim=-1).indices
            tok = best[rows, cols].gather(-1, int32(rank).long().T[..., None] % most)[..., 0]
        else:
            x = ru(N, B)
            y = t if c["draft"] == "none" else q
            tok = torch.stack([(y[rows[n], cols].cumsum(-1) < x[n, :, None]).sum(-1) for n in range(N)])
        s["token"] = tok.clamp_max(V - 1).T.contiguous().to(torch.int32)         # [B,N]
        s["parent"], s["pos"], s["u"] = parent, int32(_positions(c)), ru(N + 1, B)
        s["target"], s["target0"] = t[:N], t[N] if c["root"] else None
        s["draft"], s["draft0"] = (q[:N], q[N] if c["root"] else None) if c["draft"] != "none" else (None, None)
        P = s["P"] = min(N, c["depth"])
        s["path"] = torch.zeros((B, P), device=dev, dtype=torch.int32)
        s["n_path"], s["next"] = torch.zeros_like(s["pos"]), torch.zeros_like(s["pos"])
        if own:
            from recurrent_state_quant_lq_amd import lq
            s["dims"] = lq.make_dims(B, 1, 128, 128, c["W"], 0)
            s["work"] = torch.zeros((lq.lq_verify_workspace_bytes(s["dims"], N, V),), device=dev, dtype=torch.uint8)
        return s
    index, n = _index(c)
    s["index"], s["pos"] = int32(index), int32(_positions(c, n))
    s["pos_out"] = int32(_positions(c))
    inplace = c["kind"] in ("fork", "compact")
    s["dst"] = _states(c, B, g, dev)
    s["src"] = s["dst"] if inplace else _states(c, n, g, dev)
    if own:
        from recurrent_state_quant_lq_amd import lq
        mode = lq.LQ_DECAY_PER_KEY if c["per_key"] else lq.LQ_DECAY_SCALAR
        layers = lambda x, rows: [lq.LayerState(lq.make_dims(rows, c["H"], c["d"], c["d"], c["W"], c["C"], mode),
                                                *[x[f][i] for f in FIELDS]) for i in range(c["layers"])]
        s["dst_states"] = layers(s["dst"], B)
        s["src_states"] = s["dst_states"] if inplace else layers(s["src"], n)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "prompt":
        return _plain_prompt(s, c)
    return _plain_verify(s, c) if c["op"] == "verify" else _plain_gather(s, c)


def _moved(s):
    """The states after a gather: copies, so every code and number has to be the same."""
    return {"pos": s["pos_out"], **s["dst"]}


def _run_own(s, c):
    from recurrent_state_quant_lq_amd import lq
    if c["op"] == "prompt":
        lq.lq_gdn_prefill_ragged(s["dims"], None, s["h0"], s["h"], c["T"], s["q"], s["k"], s["v"], s["alpha"],
                                 s["beta"], s["o"], lens=s["lens"], workspace=s["work"])
        return {"o": s["o"], "h": s["h"]}
    if c["op"] == "verify":
        lq.lq_tree_verify(s["dims"], s["pos"], s["parent"], s["token"], s["target"], s["u"], s["path"], s["n_path"],
                          s["next"], target0=s["target0"], draft=s["draft"], draft0=s["draft0"],
                          replace=c["draft"] != "without", workspace=s["work"])
        return {"path": s["path"], "n_path": s["n_path"], "next": s["next"]}
    lq.lq_state_gather(s["dst_states"], s["src_states"], s["index"], s["pos"], s["pos_out"])
    return _moved(s)


def _plain_prompt(s, c):
    """Chunks: within a chunk (I + A) M = R with A strictly lower triangular, between chunks the
    state.  One token: the recurrence itself."""
    T, B, H, d = c["T"], c["B"], c["H"], c["d"]
    dev, io, per_key = s["q"].device, IO[c["io"]], c["per_key"]
    al = s["alpha"] if per_key else s["alpha"][..., None]
    if T == 1:
        k, v = s["k"][0].float(), s["v"][0].float()
        h = s["h0"] * al[0][..., None] if s["h0"] is not None else torch.zeros((B, H, d, d), device=dev)
        u = s["beta"][0][..., None] * (v - (h * k[..., None]).sum(2))
        h = h + k[..., None] * u[..., None, :]
        return {"o": (h * s["q"][0].float()[..., None]).sum(2)[None].to(io), "h": h}
    L = min(16 if per_key else CHUNK, T)
    n = -(-T // L)
    pad = n * L - T

    def chunks(x):                                       # [T,B,H,...] -> [B*H, chunks, L, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 1) + (0, pad))
        return x.reshape(n, L, B * H, -1).permute(2, 0, 1, 3).contiguous()

    real = torch.ones((T, B), device=dev, dtype=torch.bool)
    if s["lens"] is not None:
        real = torch.arange(T, device=dev)[:, None] < s["lens"][None, :]
    mask = real[:, :, None, None].expand(T, B, H, 1)
    # log decays: sums in 64 bits, since neighbours' differences count; padded tokens change nothing
    g = chunks(al.double().log() * mask).cumsum(2)       # [BH, n, L, gd]
    q, k, v = (chunks(s[x].float() * mask) for x in "qkv")
    beta = chunks(s["beta"][..., None] * mask)
    lower = torch.ones((L, L), device=dev, dtype=torch.bool).tril()
    h = s["h0"].reshape(B * H, d, d).clone() if s["h0"] is not None else torch.zeros((B * H, d, d), device=dev)
    eye = torch.eye(L, device=dev)

    def scores(i):
        """(K E K^T, Q E K^T) of chunk(s) i, on and below the diagonal."""
        ki, qi, gi = k[:, i], q[:, i], g[:, i]
        if not per_key:
            D = (gi - gi.transpose(-1, -2)).masked_fill(~lower, -math.inf).exp().float()
            kt = ki.transpose(-1, -2).contiguous()
            return torch.matmul(ki, kt) * D, torch.matmul(qi, kt) * D
        D = (gi[..., :, None, :] - gi[..., None, :, :]).masked_fill(~lower[..., None], -math.inf).exp().float()
        D = D * ki[..., None, :, :]
        return (D * ki[..., :, None, :]).sum(-1), (D * qi[..., :, None, :]).sum(-1)

    def solve(a, bt):
        """(I + A)^-1, row after row; A = beta times the scores below the diagonal."""
        A = bt * a.tril(-1)
        inv = eye.expand_as(A).clone()
        for r in range(1, L):
            inv[..., r, :] -= torch.matmul(A[..., r:r + 1, :r], inv[..., :r, :].contiguous())[..., 0, :]
        return inv

    if not per_key:                                      # every chunk's inverse at once
        every = slice(None)
        sk, sq = scores(every)
        inv = solve(sk, beta)
    o = torch.empty((B * H, n, L, d), device=dev)
    for i in range(n):
        if per_key:
            a, p = scores(i)
            ti = solve(a, beta[:, i])
        else:
            p, ti = sq[:, i], inv[:, i]
        gi = g[:, i]
        e, gl = gi.exp().float(), gi[:, -1:]
        m = torch.matmul(ti, beta[:, i] * (v[:, i] - torch.matmul(e * k[:, i], h)))
        o[:, i] = torch.matmul(e * q[:, i], h) + torch.matmul(p, m)
        kd = (gl - gi).exp().float() * k[:, i]
        h = gl.exp().float().transpose(-1, -2) * h + torch.matmul(kd.transpose(-1, -2).contiguous(), m)
    o = o.permute(1, 2, 0, 3).reshape(n * L, B, H, d)[:T]
    o = torch.where(real[:, :, None, None], o, 0.0).to(io)
    return {"o": o.contiguous(), "h": h.reshape(B, H, d, d)}


def _plain_verify(s, c):
    """All rows at once, node after node (a node's parent and its earlier siblings come before it); in
    64 bits, so that a number next to a border falls on the same side in any order of sums."""
    B, N, V, P = c["B"], c["N"], c["V"], s["P"]
    dev = s["pos"].device
    rows = torch.arange(B, device=dev)
    some = s["draft"] is not None
    f8 = lambda x: torch.full((B,), float(x), device=dev, dtype=torch.float64)
    cur = torch.full((B,), -1, device=dev, dtype=torch.int64)
    length = torch.zeros(B, device=dev, dtype=torch.int64)
    limit = (c["W"] - s["pos"].long()).clamp_max(P)
    path = torch.full((B, P), -1, device=dev, dtype=torch.int64)
    cc, S, Z, none = f8(0), f8(1), f8(1), torch.zeros(B, device=dev, dtype=torch.bool)
    gone = torch.zeros((B, V), device=dev, dtype=torch.bool)           # tokens rejected at the current node

    def after(x, x0):
        """The distribution after the current node."""
        y = x[cur.clamp_min(0), rows]
        return y if x0 is None else torch.where((cur < 0)[:, None], x0, y)

    for n in range(N):
        par, t = s["parent"][:, n].long(), s["token"][:, n].long()
        test = (par == cur) & (t >= 0) & (t < V) & (length < limit)
        t = t.clamp(0, V - 1)
        u = s["u"][n].double()
        p = after(s["target"], s["target0"])
        pt = p[rows, t].double()
        first = test & (cur < 0) if s["target0"] is None else none     # a token that is already chosen
        test = test & ~first & (S > 0) & (Z > 0)
        if some:
            q = after(s["draft"], s["draft0"])
            qt = q[rows, t].double()
            acc = test & (u * qt * S < (pt - cc * qt).clamp_min(0) * Z)
        else:
            pt = torch.where(gone[rows, t], 0.0, pt)
            acc = test & (u * S < pt)
        rej = test & ~acc
        if some:
            cc = torch.where(rej, cc + S / Z, cc)
            if c["draft"] == "without":
                Z = torch.where(rej & ~gone[rows, t], Z - qt, Z)
            S = torch.where(rej, (p.double() - cc[:, None] * q.double()).clamp_min(0).sum(-1), S)
        else:
            S = torch.where(rej, S - pt, S)
        gone[rows, t] = gone[rows, t] | rej
        acc = acc | first
        path.scatter_(1, length.clamp_max(P - 1)[:, None],
                      torch.where(acc, n, path.gather(1, length.clamp_max(P - 1)[:, None])[:, 0])[:, None])
        length = length + acc
        cur = torch.where(acc, n, cur)
        cc, S, Z = torch.where(acc, 0.0, cc), torch.where(acc, 1.0, S), torch.where(acc, 1.0, Z)
        gone = gone & ~acc[:, None]
    w = after(s["target"], s["target0"]).double()
    if some:
        left = (w - cc[:, None] * after(s["draft"], s["draft0"]).double()).clamp_min(0)
    else:
        left = w.masked_fill(gone, 0.0)
    w = torch.where((S > 0)[:, None], left, w)
    cum = w.cumsum(-1)
    total = cum[:, -1]
    at = (cum <= (s["u"][N].double() * total)[:, None]).sum(-1)
    last = (w > 0).long().mul(torch.arange(V, device=dev)).amax(-1)
    nxt = torch.where(total > 0, torch.minimum(at, last), -1)
    if s["target0"] is None:
        nxt = torch.where(cur < 0, -1, nxt)
    return {"path": path.int(), "n_path": length.int(), "next": nxt.int()}


def _plain_gather(s, c):
    idx, W = s["index"].long(), c["W"]
    take, clear, at = idx >= 0, idx == -2, idx.clamp_min(0)
    held = s["pos"].long()[at]
    live = torch.arange(W, device=idx.device)[None] < held[:, None]               # [B,W]
    for f in FIELDS:
        if f.startswith("comp") and c["C"] == 0:
            continue
        old, new = s["dst"][f], s["src"][f][:, at]
        if f.startswith("buf"):
            old.copy_(torch.where((take[:, None] & live)[:, None, :, None], new, old))
            continue
        empty = torch.zeros_like(old)
        if f == "col_scale":
            empty += 1
        if f == "comp_idx":
            empty += torch.arange(c["C"], device=idx.device, dtype=torch.int32)
        wide = (-1,) + (1,) * (old.dim() - 2)
        old.copy_(torch.where(take.view(wide), new, torch.where(clear.view(wide), empty, old)))
    s["pos_out"].copy_(torch.where(take, held, torch.where(clear, 0, s["pos_out"].long())))
    return _moved(s)


# ---------------------------------------------------------------------------
# 64 bits, from the definition: token after token, node after node, row after row
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    return {"prompt": _exact_prompt, "verify": _exact_verify, "gather": _exact_gather}[c["op"]](s, c)


def _exact_prompt(s, c):
    T, B, H, d = c["T"], c["B"], c["H"], c["d"]
    if T * B * H * d * d > 3e11:
        return None
    dev = s["q"].device
    h = s["h0"].double() if s["h0"] is not None else torch.zeros((B, H, d, d), device=dev, dtype=torch.float64)
    lens = torch.tensor(_lens(c), device=dev)
    o = torch.zeros((T, B, H, d), device=dev, dtype=torch.float64)
    for t in range(T):
        on = (lens > t)[:, None]
        # rows without a token: decay 1, beta 0
        al = torch.where(on[..., None] if c["per_key"] else on, s["alpha"][t].double(), 1.0)
        beta = torch.where(on, s["beta"][t].double(), 0.0)
        k, v = s["k"][t].double(), s["v"][t].double()
        h = h * (al[..., None] if c["per_key"] else al[..., None, None])
        u = beta[..., None] * (v - torch.matmul(k[..., None, :], h)[..., 0, :])
        h.addcmul_(k[..., None], u[..., None, :])
        o[t] = torch.where(on[..., None], torch.matmul(s["q"][t].double()[..., None, :], h)[..., 0, :], 0.0)
    return {"o": o, "h": h}


def _exact_verify(s, c):
    B, N, V, P = c["B"], c["N"], c["V"], s["P"]
    parents, tokens, pos = s["parent"].tolist(), s["token"].tolist(), s["pos"].tolist()
    u = s["u"].double().tolist()
    path, n_path, nxt = [], [], []
    for b in range(B):
        cur, line, limit = -1, [], min(P, c["W"] - pos[b])

        def start():
            p = s["target"][cur, b] if cur >= 0 else s["target0"][b] if s["target0"] is not None else None
            q = None if s["draft"] is None else s["draft"][cur, b] if cur >= 0 else \
                s["draft0"][b] if s["draft0"] is not None else None
            return (None if p is None else p.double()), (None if q is None else q.double())

        p, q = start()
        full = p
        while len(line) < limit:
            taken = None
            for n in range(N):
                t = tokens[b][n]
                if parents[b][n] != cur or not 0 <= t < V:
                    continue
                if p is None:                             # the token that is already chosen
                    taken = n
                    break
                pt = float(p[t])
                if pt > u[n][b] * (1.0 if q is None else float(q[t])):
                    taken = n
                    break
                if q is None:                             # p given that it is not t
                    p = p.clone()
                    p[t] = 0.0
                    rest = 1.0 - pt
                else:                                     # what the target has beyond the draft
                    p = (p - q).clamp_min(0.0)
                    rest = float(p.sum())
                if not rest > 1e-15:
                    p = full
                    break
                p = p / rest
                if q is not None and c["draft"] == "without":
                    q = q.clone()
                    z = 1.0 - float(q[t])
                    q[t] = 0.0
                    if not z > 1e-15:
                        break
                    q = q / z
            if taken is None:
                break
            line.append(taken)
            cur = taken
            p, q = start()
            full = p
        if p is None:
            nxt.append(-1)
        else:
            cum = p.cumsum(0)
            i = int((cum <= u[N][b] * cum[-1]).sum())
            nxt.append(min(i, int((p > 0).nonzero()[-1])))
        n_path.append(len(line))
        path.append(line + [-1] * (P - len(line)))
    dev = s["pos"].device
    t = lambda x: torch.tensor(x, device=dev, dtype=torch.int32)
    return {"path": t(path), "n_path": t(n_path), "next": t(nxt)}


def _exact_gather(s, c):
    index, _ = _index(c)
    pos, pos_out = s["pos"].tolist(), s["pos_out"].tolist()
    x, y = {f: s["dst"][f].clone() for f in FIELDS}, s["src"]
    for b, i in enumerate(index):
        for f in FIELDS:
            if f.startswith("comp") and c["C"] == 0:
                continue
            if i >= 0:
                if f.startswith("buf"):
                    x[f][:, b, :, :pos[i]] = y[f][:, i, :, :pos[i]]
                else:
                    x[f][:, b] = y[f][:, i]
            elif i == -2 and not f.startswith("buf"):
                x[f][:, b] = 1.0 if f == "col_scale" else 0
                if f == "comp_idx":
                    x[f][:, b] = torch.arange(c["C"], device=x[f].device, dtype=torch.int32)
        pos_out[b] = pos[i] if i >= 0 else 0 if i == -2 else pos_out[b]
    return {"pos": torch.tensor(pos_out, device=s["pos"].device, dtype=torch.int32), **x}
