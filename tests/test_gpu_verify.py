"""Verification of drafted trees on the GPU against the recursion in 64 bits: every path
and token has to be the reference's."""
import random

import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def tree(rng, N, bushy):
    """Parents of N nodes: -1, earlier nodes, and some entries that are no node."""
    par = []
    for n in range(N):
        x = rng.random()
        par.append(-1 if n == 0 or x < 0.1 * bushy else n - 1 if x < 1 - 0.6 * bushy else rng.randrange(n) if x < 0.95 else
                   rng.choice([-2, -7, n, n + 3]))
    return par


def case(seed, B, N, V, W=16, mode="with", root=True, bushy=1.0, scale=3.0, noise=0.7, cut=False):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    logits = scale * torch.randn(N + 1, B, V, generator=g)
    t = torch.softmax(logits, -1)
    if cut:
        t = torch.where(t >= 0.05 * t.amax(-1, keepdim=True), t, 0.0)
        t = t / t.sum(-1, keepdim=True)
    q = torch.softmax(logits + noise * torch.randn(N + 1, B, V, generator=g), -1)
    parent = [tree(rng, N, bushy) for _ in range(B)]
    token = []
    for b in range(B):
        tok = []
        for n in range(N):
            p = parent[b][n]
            row = (q if mode != "none" else t)[p if 0 <= p < n else N, b].clone()
            if mode == "without":
                for m in range(n):
                    if parent[b][m] == p and 0 <= tok[m] < V:
                        row[tok[m]] = 0.0
            x = int(torch.multinomial(row, 1, generator=g)) if float(row.sum()) > 0 else 0
            tok.append(x if rng.random() < 0.97 else rng.choice([-1, V, V + 5]))
        token.append(tok)
    pos = [rng.randint(0, W) for _ in range(B)]
    u = torch.rand(N + 1, B, generator=g)
    return dict(parent=parent, token=token, pos=pos, u=u, target=t[:N], target0=t[N] if root else None,
                draft=q[:N] if mode != "none" else None, draft0=q[N] if mode != "none" and root else None,
                replace=mode != "without", W=W)


def run(c, P=None, workspace=None, keep=None):
    N, B, V = c["target"].shape
    P = N if P is None else P
    d = lq.make_dims(B, 1, 16, 16, c["W"], 0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    f = lambda x: None if x is None else x.cuda().contiguous()
    out = keep or [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, P), (B,), (B,))]
    lq.lq_tree_verify(d, i32(c["pos"]), i32(c["parent"]), i32(c["token"]), f(c["target"]), f(c["u"]), *out,
                      target0=f(c["target0"]), draft=f(c["draft"]), draft0=f(c["draft0"]), replace=c["replace"],
                      workspace=workspace)
    torch.cuda.synchronize()
    return [x.cpu() for x in out]


def check(c, P=None):
    N, B, V = c["target"].shape
    P = N if P is None else P
    path, n_path, nxt = run(c, P)
    border = 0
    for b in range(B):
        row = lambda x: None if x is None else x[:, b]
        if not 0 <= c["pos"][b] <= c["W"]:
            assert path[b].tolist() == [77] * P and int(n_path[b]) == 77 and int(nxt[b]) == 77
            continue
        one = lambda x: None if x is None else x[b]
        want, tok, close = R.verify(c["parent"][b], c["token"][b], row(c["target"]), c["u"][:, b].tolist(),
                                    min(P, c["W"] - c["pos"][b]), one(c["target0"]), row(c["draft"]), one(c["draft0"]),
                                    c["replace"])
        if close < 1e-12:                                  # (a number on a border: either side is right)
            border += 1
            continue
        assert (path[b].tolist(), int(n_path[b]), int(nxt[b])) == (want + [-1] * (P - len(want)), len(want), tok), b
    assert border <= 1 + B // 50


@pytest.mark.parametrize("mode", ["with", "without", "none"])
@pytest.mark.parametrize("root", [True, False])
@pytest.mark.parametrize("N,V", [(1, 1), (1, 7), (2, 3), (5, 100), (8, 1000), (33, 257), (64, 4096), (64, 37), (7, 4097),
                                 (3, 20011)])
def test_trees(N, V, root, mode):
    check(case(N * 1000 + V, 13, N, V, mode=mode, root=root))


@pytest.mark.parametrize("mode", ["with", "without", "none"])
@pytest.mark.parametrize("cut", [False, True])
def test_many_siblings_that_are_rejected(mode, cut):
    """A draft far from the target: most children are rejected, several sums a row."""
    check(case(3, 24, 40, 5003, W=32, mode=mode, bushy=3.0, noise=4.0, cut=cut))
    check(case(4, 24, 16, 60, W=32, mode=mode, bushy=9.0, noise=4.0, cut=cut))
    check(case(5, 9, 16, 70001, W=32, mode=mode, bushy=4.0, noise=4.0, cut=cut))     # (first sums by a launch of their own)


@pytest.mark.parametrize("mode", ["with", "none"])
def test_a_large_vocabulary_and_many_rows(mode):
    check(case(6, 2, 4, 300007, mode=mode))
    check(case(7, 400, 3, 50, mode=mode, W=4))
    check(case(8, 256, 2, 70001, mode=mode, W=4))
    check(case(8, 5, 12, 70001, mode=mode, root=False))


def test_the_path_is_cut_at_P_and_at_the_window():
    c = case(8, 40, 12, 50, W=8, bushy=0.0, noise=0.0)     # the draft is the target: all accepted
    c["u"] = c["u"] * 0.9
    check(c, P=3)
    path, n_path, _ = run(c, P=3)
    assert n_path.tolist() == [min(3, 8 - p) if all(0 <= t < 50 for t in c["token"][b][:3]) and
                               c["parent"][b][:3] == [-1, 0, 1] else int(n_path[b]) for b, p in enumerate(c["pos"])]


def test_positions_outside_the_window_leave_a_row():
    c = case(9, 6, 4, 30)
    c["pos"] = [-1, 17, 16, 0, 1000, -5]
    check(c)


@pytest.mark.parametrize("V", [5, 5000, 70001])
def test_rows_with_nothing_left(V):
    """A target whose mask leaves nothing, one of a single token, NaN, a draft equal to the target,
    a draft that covers the target, numbers at the ends of [0, 1)."""
    N, B = 4, 8
    c = case(10, B, N, V)
    c["parent"] = [[-1, -1, -1, -1]] * B
    c["token"] = [[1, 2, 1, 0]] * B
    c["pos"] = [0] * B
    t, q = c["target0"], c["draft0"]
    t[0] = 0.0                                             # masked altogether
    t[1] = 0.0
    t[1, 3] = 1.0                                          # one token, not drafted
    t[2, :] = float("nan")
    t[3, :2] = float("nan")
    q[4] = t[4]                                            # every child accepted
    q[5] = t[5] * 2.0                                      # nothing beyond the draft
    c["u"][:, 5] = 0.9999999
    c["u"][:, 6] = 0.0
    c["u"][:, 7] = 0.99999994
    check(c)
    path, n_path, nxt = run(c)
    assert int(nxt[0]) == -1 and int(n_path[0]) == 0 and int(nxt[1]) == 3 and int(nxt[2]) == -1
    c["draft"] = c["draft0"] = None
    check(c)


def test_without_replacement_the_draft_runs_out():
    """Children that use up the whole draft, and a token drafted twice."""
    N, B, V = 4, 3, 6
    c = case(12, B, N, V, mode="without")
    c["parent"], c["pos"] = [[-1] * 4] * B, [0] * B
    c["token"] = [[0, 1, 2, 3], [0, 0, 1, 1], [2, 3, 2, 4]]
    c["draft0"][:] = 0.0
    c["draft0"][:, 0] = c["draft0"][:, 1] = 0.5            # exactly used up after two
    c["draft0"][2] = 0.25
    c["draft0"][2, :2] = 0.0
    c["target0"][:] = torch.tensor([0.0, 0.0, 0.0, 0.25, 0.25, 0.5])
    check(c)


@pytest.mark.parametrize("V", [9001, 70001])
@pytest.mark.parametrize("mode", ["without", "none"])
def test_streams_graphs_and_workspaces(mode, V):
    c = case(13, 9, 20, V, mode=mode, noise=2.0, bushy=2.0)
    N, B, V = c["target"].shape
    d = lq.make_dims(B, 1, 16, 16, 16, 0)
    want = run(c)
    need = lq.lq_verify_workspace_bytes(d, N, V)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    f = lambda x: None if x is None else x.cuda().contiguous()
    args = [i32(c["pos"]), i32(c["parent"]), i32(c["token"]), f(c["target"]), f(c["u"])]
    kw = dict(target0=f(c["target0"]), draft=f(c["draft"]), draft0=f(c["draft0"]), replace=c["replace"])
    outs = [[torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, N), (B,), (B,))] for _ in range(2)]
    ws = [torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for o, w in zip(outs, ws):
        lq.lq_tree_verify(d, *args, *o, workspace=w, stream=torch.cuda.Stream(), **kw)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x.cpu(), y) for x, y in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.lq_tree_verify(d, *args, *outs[0], workspace=ws[0], **kw)
    for r in range(3):                                     # other numbers every replay
        other = case(20 + r, 9, 20, V, mode=mode, noise=2.0, bushy=2.0)
        for x, y in zip(args, ("pos", "parent", "token", "target", "u")):
            x.copy_(other[y] if torch.is_tensor(other[y]) else torch.tensor(other[y], dtype=torch.int32))
        kw["target0"].copy_(other["target0"])
        if mode != "none":
            kw["draft"].copy_(other["draft"])
            kw["draft0"].copy_(other["draft0"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.cpu(), y) for x, y in zip(outs[0], run(other)))


def test_refusals():
    c = case(14, 3, 4, 10)
    N, B, V = c["target"].shape
    d = lq.make_dims(B, 1, 16, 16, 16, 0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    base = dict(pos=i32(c["pos"]), parent=i32(c["parent"]), token=i32(c["token"]), target=c["target"].cuda(),
                u=c["u"].cuda(), path=i32([[0] * N] * B), n_path=i32([0] * B), next=i32([0] * B),
                target0=c["target0"].cuda(), draft=c["draft"].cuda(), draft0=c["draft0"].cuda())
    lq.lq_tree_verify(d, **base)
    for kw in (dict(u=base["u"][:N]), dict(target=base["target"].bfloat16()), dict(draft=base["draft"][:, :, :9]),
               dict(draft0=None), dict(token=base["token"].long()), dict(path=base["path"][:2]), dict(next=base["next"][:2]),
               dict(target0=base["target0"].cpu()), dict(draft=None)):
        with pytest.raises(ValueError):
            lq.lq_tree_verify(d, **{**base, **kw})
    with pytest.raises(lq.LQError):
        lq.lq_tree_verify(d, **base, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
