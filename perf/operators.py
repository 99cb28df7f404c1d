"""Measured cases of the linear-attention operators over the int8 recurrent state.

Three operators, each in a plain form (elementary torch operations in fp32) and
through the library's entry points:

* ``prefill``  linear attention with a decay for each head over a prompt,
               H <- alpha H + k v^T, o = H^T q (``lq_la_prefill``); one token is
               its recurrent form over the fp32 state;
* ``decode``   the same recurrence for one token over the int8 state and its
               fp32 window buffer (``lq_la_decode_step_ragged``);
* ``tree``     every token of a drafted tree over the int8 state and its window,
               for the gated delta rule (scalar or per-key decay) or for plain
               linear attention, then the accepted path's slots appended to the
               window (``lq_gdn_tree_step`` / ``lq_la_tree_step``,
               ``lq_tree_commit``).

A state's codec: H_ij = sq_ij r_i s_j, rows idx_c replaced by cv_c (the int8 rows
there are zero); the stored byte order of sq is ``_byte_order``.
"""
import math
import random

import torch

own = False

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64      # tokens per chunk of the plain prefill


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _prefill(name, B, H, d, T, io, decay="token", ragged=False, start=True):
    return dict(name=name, op="prefill", B=B, H=H, d=d, T=T, io=io, decay=decay, ragged=ragged, start=start)


def _decode(name, B, H, d, W, C, io, decay="token", ragged=True):
    return dict(name=name, op="decode", B=B, H=H, d=d, W=W, C=C, io=io, decay=decay, ragged=ragged)


def _tree(name, rule, B, H, d, W, C, N, depth, io, decay="token", ragged=True):
    return dict(name=name, op="tree", rule=rule, B=B, H=H, d=d, W=W, C=C, N=N, depth=depth, io=io,
                decay=decay, ragged=ragged)


def listed():
    return [
        # one token of every sequence of a serving batch, over fp32 states
        _prefill("prefill one token", 64, 32, 128, 1, "bf16"),
        # a short prompt of one sequence: latency
        _prefill("prefill short prompt", 1, 16, 128, 512, "bf16", start=False),
        # one long document: few heads, many tokens
        _prefill("prefill long prompt", 1, 16, 128, 16384, "bf16", decay="head", start=False),
        # a padded batch of prompts of different lengths, continued from earlier states, fp32 tokens
        _prefill("prefill padded batch", 24, 8, 128, 1021, "f32", ragged=True),
        # a full batch of prompts
        _prefill("prefill batch", 64, 32, 128, 512, "bf16", start=False),
        # one sequence, one token: latency
        _decode("decode one sequence", 1, 16, 128, 16, 4, "bf16", ragged=False),
        # a serving batch, every sequence at its own window position
        _decode("decode batch", 256, 32, 128, 16, 4, "bf16"),
        # a small head and a short window, fp32 tokens
        _decode("decode d64 batch", 96, 12, 64, 8, 2, "f32", decay="head"),
        # a few drafted tokens for one sequence: latency
        _tree("tree one sequence", "gdn", 1, 16, 128, 16, 4, 8, 4, "bf16", ragged=False),
        # a serving batch with a drafted tree per sequence
        _tree("tree gdn batch", "gdn", 64, 32, 128, 16, 4, 32, 8, "bf16"),
        # per-key decay, odd tree size, fp32 tokens
        _tree("tree per-key batch", "kda", 32, 32, 128, 16, 4, 21, 6, "f32"),
        # plain linear attention with a decay for each head, the largest trees
        _tree("tree linear batch", "la", 64, 32, 128, 16, 4, 64, 12, "bf16", decay="head"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"prefill": work(listed()[4]), "decode": work(listed()[6]), "tree": work(listed()[11])}
    op = rng.choice(["prefill", "decode", "tree"])
    while True:
        B, H = _log_int(rng, 1, 256), _log_int(rng, 1, 64)
        d = rng.choice([16, 64, 128, 128, 128])
        io, decay = rng.choice(["f32", "bf16", "bf16"]), rng.choice(["token", "head"])
        W, C = rng.choice([4, 8, 13, 16, 16, 32]), rng.randint(0, 8)
        ragged = rng.random() < 0.7
        if op == "prefill":
            c = _prefill("", B, H, d, _log_int(rng, 1, 16384), io, decay, ragged, rng.random() < 0.5)
        elif op == "decode":
            c = _decode("", B, H, d, W, C, io, decay, ragged)
        else:
            rule = rng.choice(["gdn", "gdn", "kda", "la"])
            N = _log_int(rng, 1, 64)
            c = _tree("", rule, B, H, d, W, C, N, rng.randint(1, min(N, 16)), io,
                      decay if rule == "la" else "token", ragged)
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            del c["name"]
            return c


def _lens(c):
    """Tokens of each row of a prompt batch (from the whole length down to one)."""
    T, B = c["T"], c["B"]
    return [max(1, T - (b * 5 % B) * T // B) for b in range(B)] if c["ragged"] else [T] * B


def _positions(c, top):
    """Window positions of the rows, in [0, top]."""
    return [(7 * b + 3) % (top + 1) for b in range(c["B"])] if c["ragged"] else [c["W"] // 2] * c["B"]


def _trees(c):
    """Per row: the parents of its N nodes (-1: the last committed token; -2: no node), and the
    accepted path (the nodes from a root to the deepest node, cut at the window's end)."""
    N, W = c["N"], c["W"]
    rng = random.Random(1000 * N + c["depth"])
    shapes = []
    for _ in range(min(8, c["B"])):
        par, dep = [], []
        for n in range(N):
            p = -1 if n == 0 or rng.random() < 0.1 else n - 1 if rng.random() < 0.6 else rng.randrange(n)
            if p >= 0 and dep[p] + 1 > c["depth"]:
                p = -1
            par.append(p)
            dep.append(1 if p < 0 else dep[p] + 1)
        shapes.append(par)
    parents, paths = [], []
    for b, pos in enumerate(_positions(c, W)):
        par = list(shapes[b % len(shapes)])
        if c["ragged"]:                                   # some rows drafted fewer tokens
            keep = N - (3 * b) % (N // 2 + 1)
            par = par[:keep] + [-2] * (N - keep)
        chains = []
        for n, p in enumerate(par):
            chains.append([] if p == -2 else (chains[p] if p >= 0 else []) + [n])
        best = max(chains, key=len)
        parents.append(par)
        paths.append(best[:min(len(best), W - pos)] if b % 5 else best[:min(1, W - pos)])
    return parents, paths


def _ancestors(parents):
    """Total number of (node, ancestor) pairs and of nodes over the rows."""
    pairs = nodes = 0
    for par in parents:
        dep = []
        for p in par:
            dep.append(0 if p < 0 else dep[p] + 1)
        pairs += sum(x for x, p in zip(dep, par) if p != -2)
        nodes += sum(p != -2 for p in par)
    return pairs, nodes


def work(case):
    c = case
    B, H, d = c["B"], c["H"], c["d"]
    es = 4 if c["io"] == "f32" else 2
    if c["op"] == "prefill":
        n = sum(_lens(c)) * H
        al = 4 * n if c["decay"] == "token" else 4 * H
        by = n * 4 * d * es + al + B * H * d * d * 4 * (2 if c["start"] else 1)
        return {"bytes": by, "flops": n * 4 * d * d}
    codec = B * H * (d * d + 8 * d + c["C"] * (4 * d + 4))
    gd = d if c.get("rule") == "kda" else 1
    slot = 4 * (2 * d + gd)
    if c["op"] == "decode":
        slots = sum(_positions(c, c["W"] - 1)) * H
        by = codec + slots * slot + B * H * (4 * d * es + 4 + slot)
        return {"bytes": by, "flops": B * H * 2 * d * d + slots * 4 * d}
    parents, paths = _trees(c)
    pairs, nodes = _ancestors(parents)
    pos = _positions(c, c["W"])
    slots = sum(p for p, par in zip(pos, parents) if par[0] != -2)
    ctx = sum(p * sum(x != -2 for x in par) for p, par in zip(pos, parents)) + pairs
    rhs = 1 if c["rule"] == "la" else 2                  # products with the state: q, and k for the delta rule
    by = codec + H * (slots * slot + nodes * (4 * d * es + 4 * gd + 4 * (rhs - 1) + 4 * (d + gd)))
    by += H * sum(len(p) for p in paths) * (4 * (d + gd) + slot)
    return {"bytes": by, "flops": H * rhs * (nodes * 2 * d * d + ctx * 4 * d)}


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


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(s, device=dev, generator=g)
    ru = lambda *s: torch.rand(s, device=dev, generator=g)
    zeros = lambda s, dt=torch.float32: torch.zeros(s, device=dev, dtype=dt)
    B, H, d, io = c["B"], c["H"], c["d"], IO[c["io"]]
    # decays as trained gates give them (about 0.95 a token), or fixed per head from fast to slow
    gates = lambda *s: torch.sigmoid(3.0 - 0.5 * rn(*s))
    heads = lambda: torch.exp(-torch.exp2(-8.0 * (torch.arange(H, device=dev) + ru(H)) / H))
    int32 = lambda x: torch.tensor(x, device=dev, dtype=torch.int32)
    s = dict(case=c, io=io, d=d)
    if c["op"] == "prefill":
        T = c["T"]
        s["q"], s["k"] = _unit(rn(T, B, H, d)).to(io), _unit(rn(T, B, H, d)).to(io)
        s["v"] = rn(T, B, H, d).to(io)
        s["alpha"] = gates(T, B, H) if c["decay"] == "token" else heads()
        s["h0"] = 0.3 * rn(B, H, d, d) if c["start"] else None
        s["lens"] = int32(_lens(c)) if c["ragged"] else None
        s["h"], s["o"] = zeros((B, H, d, d)), zeros((T, B, H, d), io)
        if own:
            from recurrent_state_quant_lq_amd import lq
            s["dims"] = lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, _io_flag(lq, c))
            s["work"] = zeros((lq.lq_la_workspace_bytes(s["dims"], T),), torch.uint8)
        return s
    W, C = c["W"], c["C"]
    rule = c.get("rule", "la")
    gd = d if rule == "kda" else 1
    # the codec of a state with a few large rows
    idx = ru(B, H, d).topk(max(C, 1), dim=-1).indices.sort(dim=-1).values
    sq = (40 * rn(B, H, d, d)).round_().clamp_(-127, 127)
    if C:
        sq.scatter_(2, idx[..., None].expand(-1, -1, -1, d), 0.0)
    flat = torch.empty((B, H, d * d), device=dev, dtype=torch.int8)
    flat[..., _byte_order(d, dev).reshape(-1)] = sq.to(torch.int8).reshape(B, H, d * d)
    s["sq"], s["r"], s["s"] = flat, (0.5 + ru(B, H, d)) / 127, 0.2 + ru(B, H, d)
    s["idx"], s["cv"] = idx.to(torch.int32), 1.5 * rn(B, H, max(C, 1), d)
    # the open window: slots 0..W-1 hold tokens (only those before a row's position count)
    s["buf_k"], s["buf_m"] = _unit(rn(B, H, W, d)), 0.5 * rn(B, H, W, d)
    s["buf_g"] = gates(B, H, W, gd).log().cumsum(2)
    pos = _positions(c, W - 1 if c["op"] == "decode" else W)
    s["pos"] = int32(pos)
    lead = (B, H) if c["op"] == "decode" else (c["N"], B, H)
    s["q"], s["k"], s["v"] = _unit(rn(*lead, d)).to(io), _unit(rn(*lead, d)).to(io), rn(*lead, d).to(io)
    s["alpha"] = heads() if c["decay"] == "head" else gates(*lead, d) if rule == "kda" else gates(*lead)
    s["o"] = zeros((*lead, d), io)
    if c["op"] == "tree":
        s["beta"] = 0.1 + 0.8 * ru(*lead)
        parents, paths = _trees(c)
        P = max(1, max(len(p) for p in paths))
        s["parent"] = int32(parents)
        s["path"], s["n_path"] = int32([p + [-1] * (P - len(p)) for p in paths]), int32([len(p) for p in paths])
        s["tree_m"], s["tree_g"] = zeros((B, H, c["N"], d)), zeros((B, H, c["N"], gd))
    if own:
        from recurrent_state_quant_lq_amd import lq
        s["dims"] = lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if rule == "kda" else lq.LQ_DECAY_SCALAR,
                                 1, _io_flag(lq, c))
        s["state"] = lq.LayerState(s["dims"], s["sq"], s["r"], s["s"], s["idx"], s["cv"], s["buf_k"], s["buf_m"],
                                   s["buf_g"])
    return s


def _io_flag(lq, c):
    return lq.LQ_IO_BF16 if c["io"] == "bf16" else lq.LQ_IO_F32


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "tree": _plain_tree}[c["op"]](s, c)


def _run_own(s, c):
    from recurrent_state_quant_lq_amd import lq
    if c["op"] == "prefill":
        lq.lq_la_prefill(s["dims"], None, s["h0"], s["h"], c["T"], s["q"], s["k"], s["v"], s["alpha"], s["o"],
                         lens=s["lens"], workspace=s["work"])
        return {"o": s["o"], "h": s["h"]}
    st = s["state"]
    if c["op"] == "decode":
        if c["ragged"]:
            lq.lq_la_decode_step_ragged(st, s["pos"], s["q"], s["k"], s["v"], s["alpha"], s["o"])
        else:
            lq.lq_la_decode_step(st, c["W"] // 2, s["q"], s["k"], s["v"], s["alpha"], s["o"])
        return {"o": s["o"], "buf_k": st.buf_k, "buf_m": st.buf_m, "buf_g": st.buf_g}
    if c["rule"] == "la":
        lq.lq_la_tree_step(st, s["pos"], s["parent"], s["q"], s["k"], s["v"], s["alpha"], s["o"], s["tree_m"],
                           s["tree_g"])
    else:
        lq.lq_gdn_tree_step(st, s["pos"], s["parent"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["o"],
                            s["tree_m"], s["tree_g"])
    lq.lq_tree_commit(st, s["pos"], s["path"], s["n_path"], s["k"], s["tree_m"], s["tree_g"])
    return {"o": s["o"], "tree_m": s["tree_m"], "tree_g": s["tree_g"],
            "buf_k": st.buf_k, "buf_m": st.buf_m, "buf_g": st.buf_g}


def _plain_prefill(s, c):
    """Chunks of 64 tokens: within a chunk the decayed causal products, between chunks the state.
    One token: the recurrence itself."""
    T, B, H, d = c["T"], c["B"], c["H"], c["d"]
    dev = s["q"].device
    if T == 1:
        h = s["k"][0].float()[..., None] * s["v"][0].float()[..., None, :]
        if s["h0"] is not None:
            h += s["alpha"].expand(1, B, H)[0, :, :, None, None] * s["h0"]
        return {"o": (h * s["q"][0].float()[..., None]).sum(2)[None].to(s["io"]), "h": h}
    L = min(CHUNK, T)
    n = -(-T // L)
    pad = n * L - T

    def chunks(x):                                       # [T,B,H,...] -> [B*H, chunks, L, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 1) + (0, pad))
        return x.reshape(n, L, B * H, -1).permute(2, 0, 1, 3).contiguous()

    real = torch.ones((T, B), device=dev, dtype=torch.bool)
    if s["lens"] is not None:
        real = torch.arange(T, device=dev)[:, None] < s["lens"][None, :]
    mask = real[:, :, None].expand(T, B, H)
    # log decays: sums in 64 bits, since neighbours' differences count; padded tokens decay nothing
    la = s["alpha"].double().log().expand(T, B, H) * mask
    g = chunks(la[..., None])[..., 0].cumsum(-1)         # [BH, n, L]
    q, v = chunks(s["q"].float()), chunks(s["v"].float())
    k = chunks(s["k"].float() * mask[..., None])
    lower = torch.ones((L, L), device=dev, dtype=torch.bool).tril()
    D = (g[..., :, None] - g[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    intra = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * D, v)
    gL = g[..., -1:]
    add = torch.matmul((k * (gL - g).exp().float()[..., None]).transpose(-1, -2).contiguous(), v)
    # state before chunk i (i = n: the last): the decayed sum of the chunks before it
    ends = torch.nn.functional.pad(gL[..., 0].cumsum(-1), (1, 0))             # [BH, n + 1]
    past = torch.ones((n + 1, n), device=dev, dtype=torch.bool).tril(-1)
    E = (ends[:, :, None] - ends[:, None, 1:]).masked_fill(~past, -math.inf).exp().float()
    states = torch.matmul(E, add.reshape(B * H, n, d * d)).reshape(B * H, n + 1, d, d)
    if s["h0"] is not None:
        states += ends.exp().float()[..., None, None] * s["h0"].reshape(B * H, 1, d, d)
    before, h = states[:, :n], states[:, n]
    o = intra + torch.matmul(q * g.exp().float()[..., None], before)
    o = o.permute(1, 2, 0, 3).reshape(n * L, B, H, d)[:T]
    o = torch.where(real[:, :, None, None], o, 0.0).to(s["io"])
    return {"o": o.contiguous(), "h": h.reshape(B, H, d, d)}


def _base(s, dt=torch.float32):
    """The state that the codec stands for, [B,H,d,d]."""
    d, C = s["d"], s["case"]["C"]
    x = s["sq"][..., _byte_order(d, s["sq"].device).reshape(-1)].reshape(*s["sq"].shape[:2], d, d)
    h = x.to(dt) * s["r"].to(dt)[..., None] * s["s"].to(dt)[..., None, :]
    if C:
        h.scatter_add_(2, s["idx"][..., :C, None].long().expand(-1, -1, -1, d), s["cv"][:, :, :C].to(dt))
    return h


def _window(s, c):
    """Slots before each row's position, as a mask [B,1,W], and the last of their log decays [B,H,gd]."""
    W = c["W"]
    pos = s["pos"].long()
    live = (torch.arange(W, device=pos.device)[None, :] < pos[:, None])[:, None]
    last = s["buf_g"][torch.arange(c["B"], device=pos.device), :, (pos - 1).clamp_min(0)]
    return live, torch.where((pos > 0)[:, None, None], last, 0.0)


def _plain_decode(s, c):
    B, H, d = c["B"], c["H"], c["d"]
    hb = _base(s)
    live, last = _window(s, c)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    g = last + s["alpha"].log().expand(B, H)[..., None]
    e = (g - s["buf_g"][..., 0]).masked_fill(~live, -math.inf).exp()
    a = e * (s["buf_k"] * q[:, :, None]).sum(-1)
    m = s["buf_m"].masked_fill(~live[..., None], 0.0)
    o = (hb * (g.exp() * q)[..., None]).sum(2) + (a[..., None] * m).sum(2) + (q * k).sum(-1, keepdim=True) * v
    rows = torch.arange(B, device=q.device)
    pos = s["pos"].long()
    for name, x in (("buf_k", k), ("buf_m", v), ("buf_g", g)):
        s[name][rows, :, pos] = x
    return {"o": o.to(s["io"]), "buf_k": s["buf_k"], "buf_m": s["buf_m"], "buf_g": s["buf_g"]}


def _commit(s, c, k, tree_m, tree_g, buf_k, buf_m, buf_g):
    """Slots pos.. of each row: the nodes of its path."""
    path, pos = s["path"].long(), s["pos"].long()
    rows = torch.arange(c["B"], device=path.device)[:, None]
    at = torch.arange(c["W"], device=path.device)[None, :] - pos[:, None]     # [B,W]: place in the path
    on = ((at >= 0) & (at < s["n_path"][:, None]))[:, None, :, None]
    node = path.gather(1, at.clamp(0, path.shape[1] - 1)).clamp_min(0)
    for buf, x in ((buf_k, k.permute(1, 0, 2, 3)), (buf_m, tree_m.transpose(1, 2)), (buf_g, tree_g.transpose(1, 2))):
        buf.copy_(torch.where(on, x[rows, node].transpose(1, 2).to(buf.dtype), buf))


def _closure(parent):
    """Per row [B,N,N]: whether node i is an ancestor of node n (parents come before their children)."""
    N = parent.shape[1]
    a = (parent[..., None] == torch.arange(N, device=parent.device)).float()
    a = a + torch.eye(N, device=a.device)
    for _ in range(max(1, (N - 1).bit_length())):        # paths of doubling length
        a = (torch.matmul(a, a) > 0).float()
    return (a - torch.eye(N, device=a.device)) > 0


def _scores(x, k, e):
    """<x_n, e_{n,i} o k_i>: x [..,N,d], k [..,I,d], e [..,N,I,1] or [..,N,I,d]."""
    if e.shape[-1] == 1:
        return torch.matmul(x, k.transpose(-1, -2).contiguous()) * e[..., 0]
    return ((x[..., :, None, :] * k[..., None, :, :]) * e).sum(-1)


def _plain_tree(s, c):
    """The decode step's sums over the window and over each node's ancestors, all nodes at once:
    the ancestors' part is M = (I + A)^-1 R with A strictly lower triangular in the nodes' order."""
    B, H, N = c["B"], c["H"], c["N"]
    hb = _base(s)
    live, last = _window(s, c)
    q, k, v = (s[x].float().permute(1, 2, 0, 3).contiguous() for x in ("q", "k", "v"))   # [B,H,N,d]
    anc = _closure(s["parent"])
    here = (s["parent"] >= -1)[:, None, :, None]
    la = s["alpha"].log()
    la = la[None, :, None, None].expand(B, H, N, 1) if c["decay"] == "head" else \
        (la if la.dim() == 4 else la[..., None]).permute(1, 2, 0, 3)
    line = (anc | torch.eye(N, device=anc.device, dtype=torch.bool)).float()[:, None]
    g = last[:, :, None] + torch.matmul(line, la.contiguous())                # [B,H,N,gd]
    # decays from the window's slots and from the ancestors to each node
    ew = (g[..., :, None, :] - s["buf_g"][..., None, :, :]).masked_fill(~live[:, :, None, :, None], -math.inf).exp()
    et = (g[..., :, None, :] - g[..., None, :, :]).masked_fill(~anc[:, None, ..., None], -math.inf).exp()
    bm = s["buf_m"].masked_fill(~live[..., None], 0.0)
    o = torch.matmul(g.exp() * q, hb) + torch.matmul(_scores(q, s["buf_k"], ew), bm)
    m = v
    if c["rule"] != "la":
        beta = s["beta"].permute(1, 2, 0)[..., None]
        m = beta * (v - torch.matmul(g.exp() * k, hb) - torch.matmul(_scores(k, s["buf_k"], ew), bm))
        a = -beta * _scores(k, k, et)
        for _ in range(max(1, (N - 1).bit_length())):    # (I - a)^-1 = (I + a)(I + a^2)(I + a^4)...
            m = m + torch.matmul(a, m)
            a = torch.matmul(a, a)
    o = o + torch.matmul(_scores(q, k, et), m) + (q * k).sum(-1, keepdim=True) * m
    tree_m, tree_g = torch.where(here, m, 0.0), torch.where(here, g, 0.0)
    _commit(s, c, s["k"].float(), tree_m, tree_g, s["buf_k"], s["buf_m"], s["buf_g"])
    o = torch.where(here, o, 0.0).permute(2, 0, 1, 3).contiguous().to(s["io"])
    return {"o": o, "tree_m": tree_m, "tree_g": tree_g, "buf_k": s["buf_k"], "buf_m": s["buf_m"], "buf_g": s["buf_g"]}


# ---------------------------------------------------------------------------
# 64 bits, from the definition: the dense state, token after token
# ---------------------------------------------------------------------------

def _apply(h, x):
    """h^T x for every head: h [...,d,d], x [...,d]."""
    return torch.matmul(x[..., None, :], h)[..., 0, :]


def _rule(h, alpha, k, v, beta):
    """One token of H <- (I - beta k k^T) D H + beta k v^T (beta None: H <- D H + k v^T)."""
    h = h * alpha[..., None]
    u = v if beta is None else beta[..., None] * (v - _apply(h, k))
    return h + k[..., None] * u[..., None, :]


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    B, H, d = c["B"], c["H"], c["d"]
    f = lambda x: x.double()
    if c["op"] == "prefill":
        T = c["T"]
        h = f(s["h0"]) if s["h0"] is not None else torch.zeros((B, H, d, d), device=s["q"].device,
                                                                dtype=torch.float64)
        lens = torch.tensor(_lens(c), device=h.device)
        if T * B * H * d * d > 3e11:
            return None
        o = torch.zeros((T, B, H, d), device=h.device, dtype=torch.float64)
        for t in range(T):
            al = f(s["alpha"] if c["decay"] == "head" else s["alpha"][t]).expand(B, H)
            if c["ragged"]:
                on = lens > t                             # rows that still have a token
                h[on] = _rule(h[on], al[on][..., None], f(s["k"][t])[on], f(s["v"][t])[on], None)
                o[t, on] = _apply(h[on], f(s["q"][t])[on])
            else:
                h.mul_(al[..., None, None])
                h.addcmul_(f(s["k"][t])[..., None], f(s["v"][t])[..., None, :])
                o[t] = _apply(h, f(s["q"][t]))
        return {"o": o, "h": h}
    # the state that the codec and the open window stand for
    gd = s["buf_g"].shape[-1]
    pos = s["pos"].tolist()
    hb = _base(s, torch.float64)
    g_now = torch.zeros((B, H, gd), device=hb.device, dtype=torch.float64)
    for b, p in enumerate(pos):
        if p:
            gb = f(s["buf_g"][b, :, :p])
            g_now[b] = gb[:, -1]
            kb = f(s["buf_k"][b, :, :p]) * (gb[:, -1:] - gb).exp()
            hb[b] = g_now[b].exp()[..., None] * hb[b] + torch.matmul(kb.transpose(-1, -2).contiguous(),
                                                                     f(s["buf_m"][b, :, :p]))
    buf = {n: f(s[n]) for n in ("buf_k", "buf_m", "buf_g")}
    q, k, v, alpha = f(s["q"]), f(s["k"]), f(s["v"]), f(s["alpha"])
    if c["op"] == "decode":
        al = alpha.expand(B, H)[..., None]
        o = _apply(_rule(hb, al, k, v, None), q)
        for b, p in enumerate(pos):
            buf["buf_k"][b, :, p], buf["buf_m"][b, :, p] = k[b], v[b]
            buf["buf_g"][b, :, p] = g_now[b] + al[b].log()
        return {"o": o, **buf}
    N = c["N"]
    if N * B * H * d * d * 8 > 60e9:
        return None
    delta = c["rule"] != "la"
    z = lambda *sh: torch.zeros(sh, device=hb.device, dtype=torch.float64)
    o, tree_m, tree_g = z(N, B, H, d), z(B, H, N, d), z(B, H, N, gd)
    parents, paths = _trees(c)
    states = []
    for n in range(N):
        h_p, g_p = hb.clone(), g_now.clone()
        for m in sorted({par[n] for par in parents if par[n] >= 0}):
            on = torch.tensor([par[n] == m for par in parents], device=hb.device)
            h_p[on], g_p[on] = states[m][on], tree_g[on, :, m]
        al = alpha.expand(B, H) if c["decay"] == "head" else alpha[n]
        al = al if al.dim() == 3 else al[..., None]
        beta = f(s["beta"][n]) if delta else None
        decayed = h_p * al[..., None]
        u = beta[..., None] * (v[n] - _apply(decayed, k[n])) if delta else v[n]
        h_p = decayed + k[n][..., None] * u[..., None, :]
        on = torch.tensor([par[n] >= -1 for par in parents], device=hb.device)
        o[n, on] = _apply(h_p, q[n])[on]
        tree_m[on, :, n] = u[on]
        tree_g[on, :, n] = (g_p + al.log())[on]
        states.append(h_p)
    _commit(s, c, k, tree_m, tree_g, buf["buf_k"], buf["buf_m"], buf["buf_g"])
    return {"o": o, "tree_m": tree_m, "tree_g": tree_g, **buf}
