"""How many bits of their operands linear attention and drafted trees keep.

Queries and keys hold one channel each, no two keys the same one, so that every
output and every value of a state is a single product of a few operands, whose
64-bit value and rounding errors are known.  An operand in two bf16 parts is off by
up to 2^-16 (the second rounded) or 2^-15 (truncated); the bounds below are 2^-18.7
of a value up to one chunk, 2^-17.9 at most.

Bounds, in units of 2^-23 of the value, |g| <= 0.7 for every exponent:
  exponential of a difference of log decays: the logarithms 2 ulp each (1.4), a path
  sum in fp32 at most 8 roundings of g (2.8; prompts: one, 0.4), the product with log2(e)
  1.1, the function 1 ulp (1);                                            6.3 (prompts 3.9)
  a product with an operand in exact bf16 parts: the sum of three products  1
  a product of two fp32 values in three truncated parts: the parts left out are at
  most 2^-7 2^-15 + 2^-15 2^-7 + 2^-15 2^-15 of it (4.1), the sum of six 2.5  6.6
  every other product or scaling by an fp32 value                         0.5
  a chunk's rescaling of the state 0.5, its exponential 1 besides the shares of g above  1.5
"""
import math

import pytest
import torch

from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
IO = {"f32": (lq.LQ_IO_F32, torch.float32), "bf16": (lq.LQ_IO_BF16, torch.bfloat16)}
UNIT = 2.0 ** -23
# prompt outputs, bf16: 3.9 + 0.5 (e^g) + 1 (scores or state) + 1 (values, or the state's own update);
# trees 6.3 + 4 x 0.5 + 1 + 1; fp32: two products of split operands in place of the two exact ones
BITS = {"bf16": 11 * UNIT, "f32": 24 * UNIT}


def prompt_bits(io, T):
    """BITS and the rescalings of at most T/16 + 1 chunks (of 32 and 64 tokens at d >= 64)."""
    return BITS[io] + 0.75 * math.ceil(T / 16) * UNIT


def tree_bits(io, rule):
    """Rows scaled by a decay per key have 24 bits, whatever the tokens' type."""
    return BITS["f32" if rule == "kda" else io]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def values(g, *s, dtype=torch.float32):
    """+-[1, 2), every bit of the mantissa in use."""
    x = 1 + torch.rand(s, generator=g, dtype=torch.float64)
    return (x * torch.where(torch.rand(s, generator=g) < 0.5, -1.0, 1.0)).to(dtype)


def one_hot(at, x, d):
    """[..., d] with x at channel at."""
    out = torch.zeros(*x.shape, d, dtype=x.dtype)
    return out.scatter_(-1, at[..., None].expand(*x.shape, 1), x[..., None])


def rounded(got, ref, off, what):
    """got is the rounding to its type of a value within off of ref."""
    got = got.cpu()
    # (the bounds are rounded through fp32: 2^-24 more)
    lo, hi = ((ref + s * (off + 2.0 ** -24) * ref.abs()).to(got.dtype).double() for s in (-1, 1))
    bad = (got.double() < lo) | (got.double() > hi)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off by more than {off / UNIT:.0f} units"


def run_prefill(q, k, v, alpha, h0, io):
    T, B, H, d = q.shape
    dims = lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    o = torch.zeros((T, B, H, d), dtype=IO[io][1], device="cuda")
    h = torch.zeros((B, H, d, d), device="cuda")
    lq.lq_la_prefill(dims, None, None if h0 is None else h0.cuda(), h, T, q.cuda(), k.cuda(), v.cuda(), alpha.cuda(), o)
    torch.cuda.synchronize()
    return o, h


def earlier(g, T, *s):
    """An index i <= n for every n."""
    n = torch.arange(T).reshape(T, *[1] * len(s)).expand(T, *s)
    return torch.minimum((torch.rand((T, *s), generator=g) * (n + 1)).long(), n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(16, 16), (64, 64), (128, 64), (128, 128), (128, 4)])
@pytest.mark.parametrize("B,H", [(2, 6), (3, 50)])
def test_prompt_scores_and_state_update(B, H, d, T, io):
    """o_n = e^{g_n - g_i} <q_n, k_i> v_i for one i, h = e^{g_T - g_i} k_i v_i^T."""
    g = torch.Generator().manual_seed(d + T)
    t = IO[io][1]
    at = torch.arange(T)[:, None, None].expand(T, B, H)
    src = earlier(g, T, B, H)
    kx, qx, v = values(g, T, B, H, dtype=t), values(g, T, B, H, dtype=t), values(g, T, B, H, d, dtype=t)
    alpha = 1 - (0.64 / T) * torch.rand((T, B, H), generator=g)
    o, h = run_prefill(one_hot(src, qx, d), one_hot(at, kx, d), v, alpha, None, io)
    G = alpha.double().log().cumsum(0)
    pick = lambda x: x.double().gather(0, src)
    e = (G - G.gather(0, src)).exp()
    ref = (e * qx.double() * pick(kx))[..., None] * v.double().gather(0, src[..., None].expand(T, B, H, d))
    rounded(o, ref, prompt_bits(io, T), "o")
    rh = ((G[-1] - G).exp() * kx.double())[..., None] * v.double()                # [T,B,H,d]
    rounded(h[:, :, :T], rh.permute(1, 2, 0, 3), prompt_bits(io, T), "h")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(16, 40), (64, 64), (64, 200), (128, 64), (128, 200), (128, 3)])
@pytest.mark.parametrize("B,H", [(2, 6), (3, 50)])
def test_prompt_state(B, H, d, T, io):
    """o_n = e^{g_n} H0^T q_n for a query of one channel; keys are zero."""
    g = torch.Generator().manual_seed(d + T)
    t = IO[io][1]
    at = torch.randint(0, d, (T, B, H), generator=g)
    qx, v, h0 = values(g, T, B, H, dtype=t), values(g, T, B, H, d, dtype=t), values(g, B, H, d, d)
    alpha = 1 - (0.64 / T) * torch.rand((T, B, H), generator=g)
    o, h = run_prefill(one_hot(at, qx, d), torch.zeros((T, B, H, d), dtype=t), v, alpha, h0, io)
    G = alpha.double().log().cumsum(0)
    rows = torch.stack([h0.double().gather(2, at[n][..., None, None].expand(B, H, 1, d))[:, :, 0] for n in range(T)])
    rounded(o, (G.exp() * qx.double())[..., None] * rows, prompt_bits(io, T), "o")
    rounded(h, G[-1].exp()[..., None, None] * h0.double(), (4 + 0.75 * math.ceil(T / 16)) * UNIT, "h")


def tree_state(g, B, H, d, W, C, io, per_key, codec):
    dims = lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if per_key else lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    st = lq.LayerState.allocate(dims)
    sq = torch.randint(-127, 128, (B, H, d, d), generator=g, dtype=torch.int8) if codec else torch.zeros((B, H, d, d), dtype=torch.int8)
    r, s = values(g, B, H, d).abs() / 128, values(g, B, H, d).abs()
    idx = torch.stack([torch.randperm(d, generator=g)[:C].sort().values for _ in range(B * H)]).reshape(B, H, C)
    sq.scatter_(2, idx[..., None].expand(B, H, C, d), 0)
    cv = values(g, B, H, C, d) if codec else torch.zeros(B, H, C, d)
    st.load_codec(dict(sq=sq.numpy(), r=r.numpy(), s=s.numpy(), idx=idx.to(torch.int32).numpy(), cv=cv.numpy()))
    hb = sq.double() * r.double()[..., None] * s.double()[..., None, :]
    return st, hb.scatter_add(2, idx[..., None].expand(B, H, C, d), cv.double())


def run_tree(st, rule, pos, parent, q, k, v, alpha, beta):
    N, B, H, d = q.shape
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    o = torch.zeros((N, B, H, d), dtype=q.dtype, device="cuda")
    tm, tg = torch.zeros((B, H, N, d), device="cuda"), torch.zeros((B, H, N, st.buf_g.shape[-1]), device="cuda")
    args = [x.cuda() for x in (q, k, v, alpha)]
    if rule == "la":
        lq.lq_la_tree_step(st, i32([pos] * B), i32([parent] * B), *args, o, tm, tg)
    else:
        lq.lq_gdn_tree_step(st, i32([pos] * B), i32([parent] * B), *args, beta.cuda(), o, tm, tg)
    torch.cuda.synchronize()
    return o, tm


RULES = [(rule, io, d) for rule in ("la", "gdn", "kda") for io in ("f32", "bf16") for d in (16, 64, 128)]


@pytest.mark.parametrize("N", [13, 32, 64])
@pytest.mark.parametrize("rule,io,d", RULES)
def test_tree_state_and_window(rule, io, d, N):
    """o_n = e^{g_n} Hb^T q_n (no slots), then o_n = e^{g_n - g_c} <q_n, k_c> m_c for one slot c (no state).
    The drafted keys are zero; a chain."""
    B, H, W, C = 2, 4, 16, 3
    g = torch.Generator().manual_seed(N + d)
    t, per_key = IO[io][1], rule == "kda"
    lead = (N, B, H, d) if per_key else (N, B, H)
    qx, v = values(g, N, B, H, dtype=t), values(g, N, B, H, d, dtype=t)
    alpha, beta = 1 - (0.3 / N) * torch.rand(lead, generator=g), 0.1 + 0.8 * torch.rand((N, B, H), generator=g)
    parent, zero = list(range(-1, N - 1)), torch.zeros((N, B, H, d), dtype=t)
    G = alpha.double().log().cumsum(0)
    of = lambda x, at: x.gather(-1, at[..., None])[..., 0] if per_key else x      # the query's channel of a log decay

    st, hb = tree_state(g, B, H, d, W, C, io, per_key, True)
    at = torch.randint(0, d, (N, B, H), generator=g)
    o, _ = run_tree(st, rule, 0, parent, one_hot(at, qx, d), zero, v, alpha, beta)
    rows = torch.stack([hb.gather(2, at[n][..., None, None].expand(B, H, 1, d))[:, :, 0] for n in range(N)])
    rounded(o, (of(G, at).exp() * qx.double())[..., None] * rows, tree_bits(io, rule), "o of the state")

    st, _ = tree_state(g, B, H, d, W, 0, io, per_key, False)
    slot = torch.randint(0, W, (N, B, H), generator=g)
    ch = torch.stack([torch.randperm(d, generator=g)[:W] for _ in range(B * H)]).reshape(B, H, W)
    kx, m = values(g, B, H, W), values(g, B, H, W, d)
    bg = -(0.3 / W) * torch.rand((B, H, W, st.buf_g.shape[-1]), generator=g)
    bg = bg.cumsum(2)
    st.buf_k.copy_(one_hot(ch, kx, d)), st.buf_m.copy_(m), st.buf_g.copy_(bg)
    at = torch.stack([ch.gather(2, slot[n][..., None])[..., 0] for n in range(N)])
    o, _ = run_tree(st, rule, W, parent, one_hot(at, qx, d), zero, v, alpha, beta)
    pick = lambda x, n: x.double().gather(2, slot[n][..., None, None].expand(B, H, 1, x.shape[-1]))[:, :, 0]
    gc = torch.stack([pick(bg, n) for n in range(N)])                             # [N,B,H,gd]
    gn = bg[:, :, -1].double() + (G if per_key else G[..., None])
    e = (gn - gc).exp()
    e = e.gather(-1, at[..., None])[..., 0] if per_key else e[..., 0]
    ks = torch.stack([kx.double().gather(2, slot[n][..., None])[..., 0] for n in range(N)])
    rounded(o, (e * qx.double() * ks)[..., None] * torch.stack([pick(m, n) for n in range(N)]),
            tree_bits(io, rule), "o of the window")


@pytest.mark.parametrize("rule,io,d", RULES)
def test_tree_scores(rule, io, d):
    """o_n = e^{g_n - g_i} <q_n, k_i> m_i for one ancestor i, m_i = beta_i v_i: no key meets another; a chain."""
    B, H, W, N = 2, 4, 16, min(64, d)
    g = torch.Generator().manual_seed(d)
    t, per_key = IO[io][1], rule == "kda"
    st, _ = tree_state(g, B, H, d, W, 0, io, per_key, False)
    at = torch.arange(N)[:, None, None].expand(N, B, H)
    src = earlier(g, N, B, H)
    qx, kx, v = values(g, N, B, H, dtype=t), values(g, N, B, H, dtype=t), values(g, N, B, H, d, dtype=t)
    alpha = 1 - (0.6 / N) * torch.rand((N, B, H, d) if per_key else (N, B, H), generator=g)
    beta = 0.1 + 0.8 * torch.rand((N, B, H), generator=g)
    o, tm = run_tree(st, rule, 0, list(range(-1, N - 1)), one_hot(src, qx, d), one_hot(at, kx, d), v, alpha, beta)
    G = alpha.double().log().cumsum(0)
    if per_key:                                                                   # of the channel of the key
        gn, gi = G.gather(-1, src[..., None])[..., 0], G.gather(0, src[..., None].expand(N, B, H, d)).gather(-1, src[..., None])[..., 0]
    else:
        gn, gi = G, G.gather(0, src)
    m = v.double() if rule == "la" else beta.double()[..., None] * v.double()
    rounded(tm, m.permute(1, 2, 0, 3), UNIT, "m")
    ref = ((gn - gi).exp() * qx.double() * kx.double().gather(0, src))[..., None] * m.gather(0, src[..., None].expand(N, B, H, d))
    rounded(o, ref, tree_bits(io, rule), "o")


# ---------------------------------------------------------------------------
# log decays as sums in fp32
# ---------------------------------------------------------------------------

def sum_off(n):
    """A sum of n logarithms in fp32, relative: 2 ulp each, n additions (2^-24 each if they are rounded, 2^-23 if
    cut as a matrix instruction may)."""
    return (n + 4) * UNIT


@pytest.mark.parametrize("rule,io,d", [(r, "f32", d) for r in ("la", "gdn", "kda") for d in (16, 64, 128)])
@pytest.mark.parametrize("shape", ["chain", "binary"])
def test_tree_sums_of_strong_decays(rule, io, d, shape):
    """Log decays of 0 to -3 a token over 32 window slots and 64 nodes: the sums, and outputs that are one
    exponential of their difference each (to a window slot, then to an ancestor)."""
    B, H, W, N = 2, 3, 32, 64
    g = torch.Generator().manual_seed(d)
    per_key = rule == "kda"
    gd = d if per_key else 1
    # the window as decode steps leave it: sums in fp32, slot after slot
    steps = -3 * torch.rand((B, H, W, gd), generator=g) ** 4
    bg = steps.clone()
    for i in range(1, W):
        bg[:, :, i] = bg[:, :, i - 1] + steps[:, :, i]
    alpha = torch.exp(-3 * torch.rand((N, B, H, d) if per_key else (N, B, H), generator=g) ** 4)
    la = (alpha if per_key else alpha[..., None]).double().log()                  # [N,B,H,gd]
    parent = [n - 1 if shape == "chain" else (n - 1) // 2 if n else -1 for n in range(N)]
    path, depth = [], []
    for n, p in enumerate(parent):
        path.append(la[n] + (path[p] if p >= 0 else 0))
        depth.append(1 + (depth[p] if p >= 0 else 0))
    G = torch.stack(path) + bg[:, :, -1].double()
    off = torch.tensor([sum_off(W + x) for x in depth], dtype=torch.float64)[:, None, None, None]
    st, _ = tree_state(g, B, H, d, W, 0, io, per_key, False)
    slots = min(W, d)
    at = torch.arange(W) % d
    kx, m = values(g, B, H, W), values(g, B, H, W, d)
    kx[:, :, slots:] = 0.0                                                        # (no two keys of one channel)
    st.buf_k.copy_(one_hot(at[None, None].expand(B, H, W), kx, d)), st.buf_m.copy_(m), st.buf_g.copy_(bg)
    src = torch.randint(0, slots, (N, B, H), generator=g)
    qx, v = values(g, N, B, H), values(g, N, B, H, d)
    beta = torch.ones(N, B, H)
    zero = torch.zeros(N, B, H, d)
    o, _ = run_tree(st, rule, W, parent, one_hot(src, qx, d), zero, v, alpha, beta)
    pick = lambda x: torch.stack([x.double().gather(2, src[n][..., None, None].expand(B, H, 1, x.shape[-1]))[:, :, 0] for n in range(N)])
    last = lambda x: x.gather(-1, src[..., None])[..., 0] if per_key else x[..., 0]
    gn, gc = last(G), last(pick(bg))
    # (the window's own sums are inputs here; g_n's error and the difference's rounding, absolute in the exponent)
    lim = (off[..., 0] * gn.abs() + UNIT * (gn - gc).abs()) + BITS["f32"]
    ref = ((gn - gc).exp() * qx.double() * pick(kx[..., None])[..., 0])[..., None] * pick(m)
    near = ((o.cpu().double() - ref).abs() <= lim[..., None] * ref.abs() + 1e-30)
    assert bool(near.all()), f"{int((~near).sum())} outputs of the window"
    # nodes: ancestor or self i, a channel of its own
    if N <= d:
        chan = torch.arange(N)[:, None, None].expand(N, B, H)
        up = []
        for n in range(N):
            a = [n]
            while parent[a[-1]] >= 0:
                a.append(parent[a[-1]])
            up.append(a[int(torch.randint(0, len(a), (1,), generator=g))])
        up = torch.tensor(up)
        kx = values(g, N, B, H)
        st.buf_k.zero_()
        o, tm = run_tree(st, rule, W, parent, one_hot(up[:, None, None].expand(N, B, H), qx, d), one_hot(chan, kx, d), v, alpha, beta)
        pickc = lambda x: x.gather(-1, up[:, None, None, None].expand(N, B, H, 1))[..., 0] if per_key else x[..., 0]
        gn, gi = pickc(G), pickc(G[up])
        lim = (off[..., 0] * gn.abs() + off[up][..., 0] * gi.abs() + UNIT * (gn - gi).abs()) + BITS["f32"]
        ref = ((gn - gi).exp() * qx.double() * kx[up].double())[..., None] * v[up].double()
        near = ((o.cpu().double() - ref).abs() <= lim[..., None] * ref.abs() + 1e-30)
        assert bool(near.all()), f"{int((~near).sum())} outputs of the nodes"


def test_window_sums_of_strong_decays():
    """buf_g of 32 decode steps, alpha 0 (log decay -110) among them."""
    B, H, d, W = 2, 3, 64, 32
    g = torch.Generator().manual_seed(1)
    dims = lq.make_dims(B, H, d, d, W, 0)
    st = lq.LayerState.allocate(dims)
    z = torch.zeros(B, H, d, device="cuda")
    o = torch.zeros_like(z)
    total = torch.zeros(B, H, dtype=torch.float64)
    for n in range(W):
        alpha = torch.exp(-5 * torch.rand((B, H), generator=g) ** 4)
        alpha[1, 1] = 0.0 if n in (4, 20) else alpha[1, 1]
        lq.lq_la_decode_step(st, n, z, z, z, alpha.cuda(), o)
        total += torch.where(alpha == 0, torch.tensor(-110.0, dtype=torch.float64), alpha.double().log())
        got = st.buf_g[:, :, n, 0].cpu().double()
        assert bool(((got - total).abs() <= sum_off(n + 1) * total.abs() + 1e-30).all()), n
