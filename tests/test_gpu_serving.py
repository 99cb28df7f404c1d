"""The serving operators as they are used together: a padded batch of prompts, its states admitted to
and forked in a serving batch, drafted trees evaluated, verified and committed over several steps with
flushes between them, ended sequences compacted, against the dense recurrence in 64 bits."""
import random

import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
L, H, W, C, V, N = 2, 3, 16, 4, 50, 7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


class Model:
    """Layers whose tokens are rows of tables, and a head that turns the last layer's outputs into probabilities."""

    def __init__(self, d, per_key, io, seed):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g)
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        self.d, self.per_key, self.io = d, per_key, io
        self.q, self.k = unit(rn(L, V, H, d)).to(io).cuda(), unit(rn(L, V, H, d)).to(io).cuda()
        self.v = rn(L, V, H, d).to(io).cuda()
        self.alpha = torch.sigmoid(3 - (rn(L, V, H, d) if per_key else rn(L, V, H))).cuda()
        self.beta = torch.rand(L, V, H, generator=g).cuda()
        self.head = 6 * rn(H * d, V).cuda()

    def dims(self, B):
        return lq.make_dims(B, H, self.d, self.d, W, C, lq.LQ_DECAY_PER_KEY if self.per_key else lq.LQ_DECAY_SCALAR, 1,
                            lq.LQ_IO_BF16 if self.io == torch.bfloat16 else lq.LQ_IO_F32)

    def tokens(self, l, ids):
        """q, k, v, alpha, beta of layer l for token ids [..]."""
        return [x[l][ids].contiguous() for x in (self.q, self.k, self.v, self.alpha, self.beta)]

    def probabilities(self, o):
        return torch.softmax(o.float().flatten(-2) @ self.head, -1)


def token(h, x, i):
    """The dense recurrence over token i of x (layer tables), h [H,d,d] in 64 bits: the output and the new state."""
    q, k, v, al, be = (t[i].double() for t in x)
    h = h * (al[..., None] if al.dim() == 2 else al[:, None, None])
    u = be[:, None] * (v - (h * k[..., None]).sum(1))
    h = h + k[..., None] * u[:, None]
    return (h * q[..., None]).sum(1), h


def dense(st):
    h = torch.empty(st.dims.B, H, st.dims.dk, st.dims.dk, device="cuda")
    lq.lq_gdn_state_dequantize(st, h)
    return h.double()


def tree(rng):
    return [-1] + [rng.choice([n - 1, rng.randrange(n), -2 if n > N - 2 else n - 1]) for n in range(1, N)]


@pytest.mark.parametrize("d,per_key,io", [(128, False, torch.bfloat16), (64, True, torch.float32), (16, False, torch.float32)])
def test_prompts_forks_drafts_and_compaction(d, per_key, io):
    m = Model(d, per_key, io, d)
    rng = random.Random(d)
    g = torch.Generator(device="cuda").manual_seed(d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # ---- two prompts of different lengths ----
    T, lens = 40, [40, 23]
    ids = torch.randint(V, (T, 2), device="cuda", generator=g)
    ds, db = m.dims(2), m.dims(6)
    src, st = ([lq.LayerState.allocate(x) for _ in range(L)] for x in (ds, db))
    for l in range(L):
        x = m.tokens(l, ids)
        h, o = torch.empty(2, H, d, d, device="cuda"), torch.empty(T, 2, H, d, dtype=io, device="cuda")
        lq.lq_gdn_prefill_ragged(ds, src[l], None, h, T, *x, o, lens=i32(lens))
        for b in range(2):
            want = torch.zeros(H, d, d, dtype=torch.float64, device="cuda")
            for t in range(lens[b]):
                out, want = token(want, [y[:, b] for y in x], t)
            assert float((h[b].double() - want).abs().max()) <= R.gdn_tolerance(d) * float(want.abs().max())
    # ---- admitted, forked, one row empty, one left as it is ----
    pos = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    lq.lq_state_gather(st, src, i32([0, 1, 0, lq.LQ_ROW_CLEAR, 1, lq.LQ_ROW_KEEP]), None, pos)
    assert pos.tolist() == [0, 0, 0, 0, 0, 9]
    lq.lq_state_gather(st, st, i32([-1, -1, -1, -1, -1, 2]), None, pos)      # and row 5 from row 2
    live = list(range(6))
    ref = [dense(x) for x in st]                                            # per layer [6,H,d,d], kept in 64 bits
    assert torch.equal(ref[0][0], ref[0][2]) and torch.equal(ref[1][5], ref[1][2]) and not ref[0][3].any()
    nxt = torch.randint(V, (6,), device="cuda", generator=g).int()
    for step in range(6):
        B = 6
        parent = [tree(rng) for _ in range(B)]
        tok = torch.randint(V, (B, N), device="cuda", generator=g).int()
        tok[:, 0] = nxt.clamp_min(0)
        par, ids = i32(parent), tok.long().T
        outs, slots, toks = [], [], []
        for l in range(L):
            x = m.tokens(l, ids)
            o = torch.zeros(N, B, H, d, dtype=io, device="cuda")
            tm, tg = torch.zeros(B, H, N, d, device="cuda"), torch.zeros(B, H, N, d if per_key else 1, device="cuda")
            lq.lq_gdn_tree_step(st[l], pos, par, *x, o, tm, tg)
            outs.append(o)
            slots.append((x[1], tm, tg))
            toks.append(x)
        # every present node against the dense state along its path
        for l in range(L):
            for b in range(B):
                states = {-1: ref[l][b]}
                for n, p in enumerate(parent[b]):
                    if p not in states:
                        continue
                    out, states[n] = token(states[p], [y[:, b] for y in toks[l]], n)
                    got = outs[l][n, b].double()
                    lim = 4 * R.gdn_tolerance(d) * float(ref[l][b].abs().max() + 1) + torch.finfo(io).eps * out.abs()
                    assert bool(((got - out).abs() <= lim).all()), (step, l, b, n)
        target = m.probabilities(outs[-1])
        draft = torch.softmax(torch.randn(N, B, V, device="cuda", generator=g), -1)
        draft.scatter_(-1, tok.long().T[..., None].roll(-1, 0), 0.4)         # (tokens that the draft likes)
        draft /= draft.sum(-1, keepdim=True)
        u = torch.rand(N + 1, B, device="cuda", generator=g)
        path, n_path, nxt = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,)))
        lq.lq_tree_verify(m.dims(B), pos, par, tok, target, u, path, n_path, nxt, draft=draft)
        for l in range(L):
            lq.lq_tree_commit(st[l], pos, path, n_path, *slots[l])
        for b in range(B):
            line, want, close = R.verify(parent[b], tok[b].tolist(), target[:, b].cpu(), u[:, b].tolist(),
                                         min(N, W - int(pos[b])), None, draft[:, b].cpu())
            if close > 1e-12:
                assert (path[b, :int(n_path[b])].tolist(), int(nxt[b])) == (line, want)
            for l in range(L):
                for n in path[b, :int(n_path[b])].tolist():
                    ref[l][b] = token(ref[l][b], [y[:, b] for y in toks[l]], n)[1]
        pos = pos + n_path
        if step == 2:
            # rows 1 and 4 end: the last rows move into their places, with their open windows
            index = [-1, 5, -1, -1, lq.LQ_ROW_CLEAR, lq.LQ_ROW_CLEAR]
            before = pos.clone()
            lq.lq_state_gather(st, st, i32(index), before, pos)
            nxt = torch.where(i32(index) >= 0, nxt[i32(index).clamp_min(0).long()], nxt)
            for l in range(L):
                ref[l][1] = ref[l][5]
                ref[l][4] = ref[l][5] = 0.0
            assert pos[4:].tolist() == [0, 0] and int(pos[1]) == int(before[5])
        # windows that may not take another path are flushed: the reference goes on from what the codec holds
        full = torch.where(pos > W - 4, pos, 0).int()
        for l in range(L):
            h = torch.zeros(B, H, d, d, device="cuda")
            lq.lq_gdn_window_flush_ragged(st[l], full, h)
            now = dense(st[l])
            for b in range(B):
                if int(full[b]):
                    want = ref[l][b]
                    assert float((h[b].double() - want).abs().max()) <= 8 * R.gdn_tolerance(d) * float(want.abs().max() + 1)
                    ref[l][b] = now[b]
        pos = torch.where(full > 0, 0, pos).int()


@pytest.mark.parametrize("d,per_key", [(128, False), (64, True)])
def test_a_captured_serving_step(d, per_key):
    """Tree step, verification, commit, the position's advance and a gather in one graph, replayed with other
    tokens, trees, numbers and maps, leave the bits of the same calls without one."""
    io = torch.bfloat16
    m = Model(d, per_key, io, 3)
    B = 5
    dm = m.dims(B)
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    h = 0.3 * torch.randn(B, H, d, d, device="cuda", generator=g)

    class Step:
        def __init__(self):
            self.st = lq.LayerState.allocate(dm)
            lq.lq_gdn_state_quantize(self.st, h)
            self.pos, self.par, self.tok, self.index = i32(B), i32(B, N), i32(B, N), i32(B)
            self.x = [t.contiguous() for t in m.tokens(0, torch.zeros(N, B, dtype=torch.long, device="cuda"))]
            self.target, self.u = torch.ones(N, B, V, device="cuda") / V, torch.zeros(N + 1, B, device="cuda")
            self.o = torch.zeros(N, B, H, d, dtype=io, device="cuda")
            self.tm, self.tg = torch.zeros(B, H, N, d, device="cuda"), torch.zeros(B, H, N, d if per_key else 1, device="cuda")
            self.path, self.n_path, self.next, self.moved = i32(B, N), i32(B), i32(B), i32(B)
            self.ws = torch.empty(lq.lq_verify_workspace_bytes(dm, N, V), dtype=torch.uint8, device="cuda")

        def run(self):
            lq.lq_gdn_tree_step(self.st, self.pos, self.par, *self.x, self.o, self.tm, self.tg)
            lq.lq_tree_verify(dm, self.pos, self.par, self.tok, self.target, self.u, self.path, self.n_path, self.next,
                              workspace=self.ws)
            lq.lq_tree_commit(self.st, self.pos, self.path, self.n_path, self.x[1], self.tm, self.tg)
            self.moved.copy_(self.pos + self.n_path)
            lq.lq_state_gather(self.st, self.st, self.index, self.moved, self.pos)

    a, b = Step(), Step()
    for s in (a, b):
        s.index.fill_(-1)
        s.pos.fill_(W)                                     # (nothing happens)
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    rng = random.Random(2)
    for r in range(5):
        parent = torch.tensor([tree(rng) for _ in range(B)], dtype=torch.int32)
        tok = torch.randint(V, (B, N), device="cuda", generator=g).int()
        x = m.tokens(0, tok.long().T)
        target = torch.softmax(3 * torch.randn(N, B, V, device="cuda", generator=g), -1)
        target.scatter_(-1, tok.long().T[..., None].roll(-1, 0), 1.0)
        target /= target.sum(-1, keepdim=True)
        u = torch.rand(N + 1, B, device="cuda", generator=g)
        index = torch.tensor([rng.choice([b0, rng.randrange(B)]) for b0 in range(B)], dtype=torch.int32)
        for s in (a, b):
            if r == 0:
                s.pos.zero_()
            for t, y in ((s.par, parent), (s.tok, tok), (s.target, target), (s.u, u), (s.index, index), *zip(s.x, x)):
                t.copy_(y)
        torch.cuda.synchronize()
        a.run()
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.n_path.sum()) > 0 or r > 2
        for f in ("o", "tm", "tg", "path", "n_path", "next", "pos"):
            assert torch.equal(getattr(a, f), getattr(b, f)), (r, f)
        for f in ("sq", "row_scale", "comp_val", "buf_k", "buf_m", "buf_g"):
            assert torch.equal(getattr(a.st, f), getattr(b.st, f)), (r, f)
