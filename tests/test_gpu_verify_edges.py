"""Verification of drafted trees where the target's residual runs empty, against the header's
rule in 64 bits (written apart from serving_reference.verify, which leaves such rows without a token)."""
import pytest
import torch

from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
BELOW_ONE = 1.0 - 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def rule(parent, token, target, u, limit, target0, draft=None, draft0=None, replace=True):
    """One row: the path, the next token, and the relative distance of the nearest decision."""
    wide = lambda x: torch.nan_to_num(x.double(), nan=0.0)
    V, path, cur, close = target.shape[1], [], -1, 1.0
    while True:
        p = wide(target0 if cur < 0 else target[cur])
        q = None if draft is None else wide(draft0 if cur < 0 else draft[cur])
        c, S, Z, out, taken, rejected = 0.0, 1.0, 1.0, set(), None, False
        left = lambda: (p - c * q).clamp_min(0.0) if q is not None else \
            p.index_fill(0, torch.tensor(sorted(out), dtype=torch.long), 0.0)
        for n, t in enumerate(token):
            if parent[n] != cur or n <= cur or not 0 <= t < V or len(path) >= limit or S <= 0 or Z <= 0:
                continue
            has = max(float(p[t]) - c * float(q[t]), 0.0) * Z if q is not None else 0.0 if t in out else float(p[t])
            asks = u[n] * (1.0 if q is None else float(q[t])) * S
            if has > 0:
                close = min(close, abs(has - asks) / max(has, asks))
            if asks < has:
                taken = n
                break
            rejected = True
            if q is None:
                S -= 0.0 if t in out else float(p[t])
            else:
                c, Z = c + S / Z, Z - (0.0 if replace or t in out else float(q[t]))
                S = float(left().sum())
            out.add(t)
        if taken is None:
            w = left() if rejected and S > 0 else p
            if not float(w.sum()) > 0:
                w = p
            cum = w.cumsum(0)
            if not float(cum[-1]) > 0:
                return path, -1, close
            theta = u[len(token)] * float(cum[-1])
            nxt = min(int((cum <= theta).sum()), int((w > 0).nonzero()[-1]))
            return path, nxt, min(close, float((cum - theta).abs().min()) / float(cum[-1]))
        path.append(taken)
        cur = taken


def run(B, V, N, parent, token, u, target, target0, draft=None, draft0=None, replace=True):
    """The same tree for B rows; target0 etc. [V] for all rows or [B,V], target [N,V] or [N,B,V]."""
    d = lq.make_dims(B, 1, 16, 16, 16, 0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).expand(B, -1).contiguous().cuda()
    rows = lambda x: None if x is None else x.expand(B, V).contiguous().cuda()
    after = lambda x: None if x is None else x[:, None].expand(N, B, V).contiguous().cuda()
    out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,))]
    lq.lq_tree_verify(d, torch.zeros(B, dtype=torch.int32, device="cuda"), i32(parent), i32(token), after(target),
                      torch.tensor(u).float()[:, None].expand(N + 1, B).contiguous().cuda(), *out, target0=rows(target0),
                      draft=after(draft), draft0=rows(draft0), replace=replace)
    torch.cuda.synchronize()
    return [x.cpu() for x in out]


def check(V, parent, token, u, target, target0, draft=None, draft0=None, replace=True):
    N = len(token)
    u = [float(torch.tensor(x).float()) for x in u]
    path, nxt, close = rule(parent, token, target, u, N, target0, draft, draft0, replace)
    for B in (3, 300):                                     # (few large rows by two launches, many by one)
        got = run(B, V, N, parent, token, u, target, target0, draft, draft0, replace)
        assert close > 1e-12 or draft is None              # (without a draft the kernel's tests are these operations)
        for b in range(B):
            assert (got[0][b].tolist(), int(got[1][b]), int(got[2][b])) == (path + [-1] * (N - len(path)), len(path), nxt), \
                (B, b, path, nxt)
    return path, nxt


SMALL = [(0.5, 0.49999997), (0.99827576, 0.00134207, 0.00038210), (0.99999994,), (0.3, 0.2, 0.25, 0.24999997)]


@pytest.mark.parametrize("V", [4, 5003, 70001])
@pytest.mark.parametrize("values", SMALL)
@pytest.mark.parametrize("at_end", [0.0, 0.3, 0.7, BELOW_ONE])
def test_a_whole_support_that_is_rejected_without_a_draft(values, V, at_end):
    """Probabilities that sum to a little less than 1, every token of them looked up and rejected: the
    next token comes from the target itself, at the first node and at a later one."""
    tokens = [x for x in range(V - 1, -1, -max(1, V // 5))][:len(values)]
    p = torch.zeros(V)
    p[tokens] = torch.tensor(values)
    left = 1.0 - sum(float(x) for x in p[tokens].double())
    assert 0 < left < 1e-6
    none = torch.zeros(V)
    # u: the last numbers below 1 but where a smaller one already rejects
    u, S = [], 1.0
    for t in tokens:
        u.append(min(BELOW_ONE, (float(p[t]) / S + BELOW_ONE) / 2 if float(p[t]) < 0.9 * S else BELOW_ONE))
        S -= float(p[t])
    N = len(tokens)
    assert u[-1] * (S + float(p[tokens[-1]])) >= float(p[tokens[-1]])      # (the last token is rejected too)
    path, nxt = check(V, [-1] * N, tokens, u + [at_end], none.expand(N, V), p)
    assert path == [] and nxt in tokens
    sure = torch.zeros(V)
    sure[1] = 1.0
    path, nxt = check(V, [-1] + [0] * N, [1] + tokens, [0.5] + u + [at_end],
                      torch.stack([p] + [none] * N), sure)
    assert path == [0] and nxt in tokens


NAN = float("nan")


@pytest.mark.parametrize("V", [4, 5003, 70001])
def test_nan_at_a_child_counts_as_zero(V):
    """The child with NaN is rejected and changes nothing for the ones after it, nor for the draw."""
    p, q = torch.zeros(V), torch.full((V,), 0.25 / V)
    p[:4] = torch.tensor([0.1, NAN, 0.6, 0.3])
    none = torch.zeros(2, V)
    assert check(V, [-1, -1], [1, 2], [0.2, 0.2, 0.5], none, p)[0] == [1]
    path, nxt = check(V, [-1, -1], [1, 2], [0.2, 0.9, 0.3], none, p)      # both rejected: 2 is not drawn
    assert (path, nxt) == ([], 3)
    q[1], q[2] = NAN, 0.5
    for replace in (True, False):
        p[1] = 0.0
        assert check(V, [-1, -1], [1, 2], [0.2, 0.2, 0.5], none, p, none, q, replace)[0] == [1]
        p[1] = 0.01                                        # more than none: accepted
        assert check(V, [-1, -1], [1, 2], [0.99, 0.2, 0.5], none, p, none, q, replace)[0] == [0]
    q[2], q[3] = 0.9, NAN                                  # its whole share stays after a rejection
    assert check(V, [-1], [2], [0.99, 0.4], none[:1], p, none[:1], q) == ([], 3)


@pytest.mark.parametrize("mode", ["with", "without", "none"])
@pytest.mark.parametrize("V", [7, 5003, 70001])
@pytest.mark.parametrize("seed", range(6))
def test_nan_anywhere_counts_as_zero(seed, V, mode):
    """A third of both distributions NaN, drafted tokens among them; siblings and a chain."""
    g = torch.Generator().manual_seed(100 * seed + V)
    N = 8
    logits = 2.0 * torch.randn(N + 1, V, generator=g)
    spoil = lambda x: torch.where(torch.rand(x.shape, generator=g) < 0.33, NAN, x)
    t, q = spoil(torch.softmax(logits, -1)), spoil(torch.softmax(logits + 2.0 * torch.randn(N + 1, V, generator=g), -1))
    parent = [-1, -1, -1, 0, 0, 1, 2, 2] if seed % 2 else [-1] * N
    token = [int(torch.topk(torch.nan_to_num(t[N] if n < 3 else q[N]), 4).indices[n % 4]) if n % 3 else
             int(torch.randint(V, (1,), generator=g)) for n in range(N)]
    u = (torch.rand(N + 1, generator=g) * (1.0 if seed < 3 else 0.1)).tolist()
    d = dict(draft=q[:N], draft0=q[N], replace=mode == "with") if mode != "none" else {}
    check(V, parent, token, u, t[:N], t[N], **d)
