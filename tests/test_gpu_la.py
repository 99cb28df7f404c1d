"""Linear attention with a decay per head (prompt, single token) and drafted
token trees on the GPU, against 64-bit references whose error bounds come from
the formulas (la_reference.py)."""
import pytest
import torch

import la_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
IO = {"f32": (lq.LQ_IO_F32, torch.float32), "bf16": (lq.LQ_IO_BF16, torch.bfloat16)}
MARK = 12345.0       # what untouched rows hold


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    uni = lambda *s: torch.rand(s, generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    return rnd, uni, unit


def near(got, ref, bound, what, dtype=torch.float32):
    """|got - ref| <= bound, plus half a step of the output's type."""
    got = got.double().cpu()
    lim = bound.cpu() + R.half_step(dtype) * (ref.abs().cpu() + bound.cpu()) + 1e-37
    off = (got - ref.cpu()).abs()
    worst = float((off / lim).max())
    assert bool((off <= lim).all()), f"{what}: {worst:.2f} times the bound"


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------

def prefill_case(seed, B, H, d, T, io, heads=False, start=True, scale=1.0):
    rnd, uni, unit = gen(seed)
    t = IO[io][1]
    q, k = unit(rnd(T, B, H, d)).to(t), unit(rnd(T, B, H, d)).to(t)
    v = rnd(T, B, H, d).to(t)
    alpha = (0.2 + 0.8 * uni(H)) if heads else torch.sigmoid(3.0 - scale * rnd(T, B, H))
    h0 = 0.3 * rnd(B, H, d, d) if start else None
    return q, k, v, alpha, h0


def run_prefill(q, k, v, alpha, h0, io, lens=None, st=None, o=None, with_o=True, ws=True):
    T, B, H, d = q.shape
    dims = lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    dev = lambda x: None if x is None else x.cuda().contiguous()
    if o is None and with_o:
        o = torch.full((T, B, H, d), MARK, dtype=IO[io][1], device="cuda")
    h = torch.full((B, H, d, d), MARK, device="cuda")
    need = lq.lq_la_workspace_bytes(dims, T)
    w = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") if need and ws else None   # garbage: NaN bits
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    lq.lq_la_prefill(dims, st, dev(h0), h, T, dev(q), dev(k), dev(v), dev(alpha), o, lens=lens, workspace=w)
    torch.cuda.synchronize()
    return o, h


def check_prefill(o, h, q, k, v, alpha, h0, io, lens=None, what=""):
    """Bounds: c(d) and the rescalings along a prompt, 2 per 16 tokens; a decay's logarithm and
    exponential are off by 2^-24 of an argument that matters up to 16 and by the function's 2 ulp,
    inside c(d).  bf16 outputs: products that reach o only keep 16 bits of an operand (2^-16)."""
    lt = None if lens is None else torch.tensor(lens)
    cu = lambda x: None if x is None else x.cuda()
    ro, rh, oa, ha = R.la_prefill(cu(q), cu(k), cu(v), cu(alpha), cu(h0), lt)
    T, d = q.shape[0], q.shape[-1]
    c = R.c_of(d) + 2 * (T / 16 + 1) * R.U
    near(h, rh, c * ha, what + " h")
    if o is not None:
        co = c + (2.0 ** -16 if io == "bf16" else 0.0)
        real = torch.ones(T, q.shape[1], dtype=torch.bool) if lens is None else torch.arange(T)[:, None] < lt[None]
        near(o.cpu()[real], ro.cpu()[real], co * oa.cpu()[real], what + " o", IO[io][1])
        assert bool((o.cpu()[~real].float() == torch.tensor(MARK, dtype=IO[io][1]).float()).all()), "rows past a length"


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130])
def test_prefill_lengths(T, d, io):
    c = prefill_case(T * 100 + d, 2, 3, d, T, io, heads=T % 2 == 0, start=T % 3 != 0)
    o, h = run_prefill(*c, io)
    check_prefill(o, h, *c, io)


@pytest.mark.parametrize("B,H,d,T,io", [(1, 1, 128, 1500, "bf16"), (1, 2, 128, 2049, "f32"), (3, 1, 64, 1111, "bf16"),
                                        (1, 1, 64, 900, "f32"), (1, 3, 16, 1300, "bf16"), (2, 1, 16, 777, "f32"),
                                        (1, 16, 128, 4096, "bf16"), (1, 1, 128, 20001, "bf16")])
def test_prefill_long_prompts_of_few_heads(B, H, d, T, io):
    c = prefill_case(T, B, H, d, T, io)
    o, h = run_prefill(*c, io)
    check_prefill(o, h, *c, io)


@pytest.mark.parametrize("B,H,d,T,io", [(40, 33, 128, 40, "bf16"), (10, 13, 128, 200, "f32"), (13, 10, 128, 300, "bf16"),
                                        (129, 1, 64, 150, "f32"), (64, 2, 64, 150, "bf16"), (150, 30, 16, 40, "bf16")])
def test_prefill_many_heads(B, H, d, T, io):
    c = prefill_case(5, B, H, d, T, io, heads=True, start=False)
    o, h = run_prefill(*c, io)
    check_prefill(o, h, *c, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_more_heads_than_a_chunk_takes(io):
    """Above 2^17 heads the recurrence itself runs, whatever the length (two groups of tokens and one token)."""
    c = prefill_case(6, 1025, 128, 16, 9, io)
    lens = [(5 * b) % 10 for b in range(1025)]
    o, h = run_prefill(*c, io, lens=lens)
    check_prefill(o, h, *c, io, lens=lens)


@pytest.mark.parametrize("T", [3, 40, 1300])
def test_prefill_rows_without_tokens_and_without_a_start(T):
    """A row of length 0 from zeros ends with zeros; its o rows stay."""
    c = prefill_case(T, 2, 2, 128, T, "bf16", start=False)
    o, h = run_prefill(*c, "bf16", lens=[0, T])
    check_prefill(o, h, *c, "bf16", lens=[0, T])
    assert float(h[0].abs().max()) == 0.0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(128, 70), (64, 70), (16, 70), (128, 1400), (64, 1400), (16, 1400), (128, 3)])
def test_prefill_padded_rows(d, T, io):
    """Tokens past a row's length may hold NaN; their o rows stay; rows without tokens keep h0."""
    q, k, v, alpha, h0 = prefill_case(7 * d + T, 7, 2, d, T, io)
    lens = [T, 0, 1, T - 1, -4, T + 9, T // 2]
    real = torch.arange(T)[:, None] < torch.tensor(lens)[None]
    clean = (q, k, v, alpha, h0)
    q, k, v = (torch.where(real[..., None, None], x, float("nan")).to(x.dtype) for x in (q, k, v))
    alpha = torch.where(real[..., None], alpha, float("nan"))
    o, h = run_prefill(q, k, v, alpha, h0, io, lens=lens)
    lens = [min(max(x, 0), T) for x in lens]
    check_prefill(o, h, *clean, io, lens=lens)
    assert torch.equal(h[1].cpu(), h0[1]) and torch.equal(h[4].cpu(), h0[4])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 1300])
def test_prefill_forgets_and_keeps(T, io):
    """alpha = 0 drops everything before the token, alpha = 1 keeps it, tiny alphas do not overflow."""
    q, k, v, alpha, h0 = prefill_case(T, 1, 4, 128, T, io)
    alpha[:, :, 1] = 1.0
    alpha[::5, :, 2] = 0.0
    alpha[3::7, :, 3] = 1e-38
    alpha[4::7, :, 3] = 1e-20
    o, h = run_prefill(q, k, v, alpha, h0, io)
    check_prefill(o, h, q, k, v, alpha, h0, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(128, 50), (64, 50), (16, 50), (128, 1200), (128, 6)])
def test_prefill_nonfinite_values_reach_their_column_from_their_token(d, T, io):
    q, k, v, alpha, h0 = prefill_case(T + d, 1, 2, d, T, io)
    alpha = alpha.clamp(min=0.5)
    clean = v.clone()
    bad = T // 2 + 1
    v[bad, 0, 0, 5] = float("inf")
    v[bad + 1, 0, 1, 9] = float("nan")
    o, h = run_prefill(q, k, v, alpha, h0, io)
    o, h = o.cpu().float(), h.cpu()
    assert not torch.isfinite(o[bad, 0, 0, 5]) and torch.isnan(o[bad + 1:, 0, 1, 9]).all()
    assert not torch.isfinite(h[0, 0, :, 5]).any() and not torch.isfinite(h[0, 1, :, 9]).any()
    ro, rh, oa, ha = R.la_prefill(q, k, clean, alpha, h0)
    ok_o, ok_h = torch.ones_like(o, dtype=torch.bool), torch.ones_like(h, dtype=torch.bool)
    ok_o[bad:, 0, 0, 5] = ok_o[bad + 1:, 0, 1, 9] = False
    ok_h[0, 0, :, 5] = ok_h[0, 1, :, 9] = False
    assert torch.isfinite(o[ok_o]).all() and torch.isfinite(h[ok_h]).all()
    c = R.c_of(d) + 2 * (T / 16 + 1) * R.U
    near(o[ok_o], ro[ok_o], ((c + (2.0 ** -16 if io == "bf16" else 0)) * oa)[ok_o], "o", IO[io][1])
    near(h[ok_h], rh[ok_h], (c * ha)[ok_h], "h")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(128, 50), (64, 50), (16, 50), (128, 1200), (16, 1200), (128, 4)])
def test_prefill_nonfinite_queries_and_keys_reach_nothing_before_them(d, T, io):
    """A query's reaches its own output only; a key's reaches the outputs from its token on."""
    q, k, v, alpha, h0 = prefill_case(3 * T + d, 1, 3, d, T, io)
    at = min(T - 2, 37 if T < 100 else 1001)
    bad_q, bad_k = q.clone(), k.clone()
    bad_q[at, 0, 0, 3], bad_q[at, 0, 1, 2] = float("inf"), float("nan")
    bad_k[at, 0, 2, 5] = float("nan")
    o, h = run_prefill(bad_q, bad_k, v, alpha, h0, io)
    assert not torch.isfinite(o[at, 0, :2]).any() and torch.isnan(o[at:, 0, 2]).all() and torch.isnan(h[0, 2, 5]).all()
    o2, h2 = run_prefill(q, k, v, alpha, h0, io)
    check_prefill(o2, h2, q, k, v, alpha, h0, io)
    fine = torch.ones(T, 1, 3, dtype=torch.bool, device="cuda")
    fine[at, 0, :2], fine[at:, 0, 2] = False, False
    assert torch.equal(o[fine], o2[fine]) and torch.equal(h[0, :2], h2[0, :2])


@pytest.mark.parametrize("T", [0, 1, 70, 1100])
def test_prefill_in_place_without_outputs_and_codec(T):
    """h may be h0; o may be left out; the codec written is that of the h written; T = 0 copies h0."""
    c = prefill_case(T + 3, 2, 2, 128, T, "f32")
    q, k, v, alpha, h0 = c
    dims = lq.make_dims(2, 2, 128, 128, 16, 4)
    need = lq.lq_la_workspace_bytes(dims, T)
    w = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    st, st2 = lq.LayerState.allocate(dims), lq.LayerState.allocate(dims)
    h = h0.cuda()
    dev = [x.cuda() for x in (q, k, v, alpha)]
    lq.lq_la_prefill(dims, st, h, h, T, *dev, None, workspace=w)
    o2, h2 = run_prefill(*c, "f32")
    assert torch.equal(h, h2)
    if T == 0:
        assert torch.equal(h.cpu(), h0)
        z = torch.full_like(h, MARK)
        lq.lq_la_prefill(dims, None, None, z, 0, None, None, None, None)
        assert float(z.abs().max()) == 0.0
    lq.lq_gdn_state_quantize(st2, h)
    for f in ("sq", "row_scale", "col_scale", "comp_idx", "comp_val"):
        assert torch.equal(getattr(st, f), getattr(st2, f)), f
    # the binding's own workspace, on a side stream
    h3 = h0.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lq.lq_la_prefill(dims, None, h3, h3, T, *dev, None, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(h3, h)


def test_prefill_split_in_two_calls():
    """A prompt in two calls (the second continues from the first's state) equals one call to rounding."""
    c = prefill_case(31, 1, 2, 128, 1000, "f32")
    q, k, v, alpha, h0 = c
    o, h = run_prefill(*c, "f32")
    oa, ha = run_prefill(q[:333], k[:333], v[:333], alpha[:333], h0, "f32")
    ob, hb = run_prefill(q[333:], k[333:], v[333:], alpha[333:], ha.cpu(), "f32")
    check_prefill(torch.cat([oa, ob]), hb, *c, "f32")


def test_prefill_refusals():
    dims = lq.make_dims(1, 16, 128, 128, 16, 4)
    T = 8192
    need = lq.lq_la_workspace_bytes(dims, T)
    x = torch.zeros((T, 1, 16, 128), device="cuda")
    al, h = torch.ones((T, 1, 16), device="cuda"), torch.zeros((2, 16, 128, 128), device="cuda")
    if need:
        with pytest.raises(lq.LQError):
            lq.lq_la_prefill(dims, None, None, h[:1], T, x, x, x, al, x,
                             workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):                       # overlapping states
        lq.lq_la_prefill(dims, None, h.view(-1)[128:128 + 16 * 16384].view(1, 16, 128, 128), h[:1], 1, x[:1], x[:1],
                         x[:1], al[:1], x[:1])
    with pytest.raises(ValueError):
        lq.lq_la_prefill(dims, None, None, h[:1], T, x, x, x, al[:, :, :5], x)
    with pytest.raises(ValueError):
        lq.lq_la_prefill(dims, None, None, h[:1], T, x, x, x.transpose(0, 1), al, x)


# ---------------------------------------------------------------------------
# the int8 state
# ---------------------------------------------------------------------------

def make_state(seed, B, H, d, W, C, io, per_key=False, slots=None):
    """A layer whose codec and first `slots` window slots hold values; the other slots NaN."""
    rnd, uni, unit = gen(seed)
    dims = lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if per_key else lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    st = lq.LayerState.allocate(dims)
    h = rnd(B, H, d, d)
    h[:, :, ::7] *= 6.0
    lq.lq_gdn_state_quantize(st, h.cuda())
    gd = d if per_key else 1
    bk, bm = unit(rnd(B, H, W, d)), rnd(B, H, W, d)
    bg = (0.02 + 0.3 * uni(B, H, W, gd)).neg().cumsum(2)
    if slots is not None:
        dead = torch.arange(W)[None] >= torch.tensor(slots)[:, None]
        for x in (bk, bm, bg):
            x.masked_fill_(dead[:, None, :, None], float("nan"))
    st.buf_k.copy_(bk), st.buf_m.copy_(bm), st.buf_g.copy_(bg)
    cd = st.codec()
    t = lambda a: torch.from_numpy(a)
    hb = R.dequantize(t(cd["sq"]), t(cd["r"]), t(cd["s"]), t(cd["idx"]), t(cd["cv"]))
    return dims, st, hb, bk, bm, bg


def tokens(seed, lead, d, io, per_key=False, heads=None):
    rnd, uni, unit = gen(seed)
    t = IO[io][1]
    q, k = unit(rnd(*lead, d)).to(t), unit(rnd(*lead, d)).to(t)
    v = rnd(*lead, d).to(t)
    alpha = 0.3 + 0.7 * (uni(heads) if heads else uni(*lead, d) if per_key else uni(*lead))
    beta = 0.05 + 0.9 * uni(*lead)
    return q, k, v, alpha, beta


def one_token(st, pos, q, k, v, alpha, o):
    lq.lq_la_decode_step_ragged(st, torch.tensor(pos, dtype=torch.int32).cuda(), q.cuda(), k.cuda(), v.cuda(),
                                alpha.cuda(), o)
    torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,W,C", [(128, 16, 4), (128, 32, 8), (128, 4, 0), (128, 13, 1), (64, 16, 4), (64, 32, 0),
                                   (64, 7, 8), (16, 4, 1), (16, 32, 8), (16, 16, 0)])
def test_decode_step(d, W, C, io):
    """Every position of the window at once (one row each), two rows outside it."""
    pos = list(range(W)) + [-1, W]
    B, H = len(pos), 3
    dims, st, hb, bk, bm, bg = make_state(d + W, B, H, d, W, C, io, slots=[max(p, 0) for p in pos])
    heads = H if W % 2 else None
    q, k, v, alpha, _ = tokens(W, (B, H), d, io, heads=heads)
    o = torch.full((B, H, d), MARK, dtype=IO[io][1], device="cuda")
    one_token(st, pos, q, k, v, alpha, o)
    tree_pos = [p if 0 <= p < W else -1 for p in pos]
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, tree_pos, [[-1]] * B, q[None], k[None], v[None],
                                      alpha if heads else alpha[None])
    on = here[:, 0]
    near(o.cpu()[on], ro[0][on], eo[0][on], "o", IO[io][1])
    mark = torch.tensor(MARK, dtype=IO[io][1]).float()
    assert bool((o.cpu()[~on].float() == mark).all())
    for b, p in enumerate(pos):
        if not on[b]:
            continue
        assert torch.equal(st.buf_k[b, :, p].cpu(), k[b].float()) and torch.equal(st.buf_m[b, :, p].cpu(), v[b].float())
        near(st.buf_g[b, :, p], rg[b, :, 0], 8 * R.U * (rg[b, :, 0].abs() + 1), "g")
    # nothing else of the window moved
    keep = torch.ones(B, W, dtype=torch.bool)
    for b, p in enumerate(pos):
        if on[b]:
            keep[b, p] = False
    for name, x in (("buf_k", bk), ("buf_m", bm), ("buf_g", bg)):
        got = getattr(st, name).cpu().transpose(1, 2)[keep]
        assert torch.equal(got.nan_to_num(7.0), x.transpose(1, 2)[keep].nan_to_num(7.0)), name
    # the lockstep call writes the same
    if W == 16:                                       # (a row of the state as a view: 16-byte aligned for these)
        p = W - 1
        st1 = st.rows(p, p + 1)
        o1 = torch.zeros((1, H, d), dtype=IO[io][1], device="cuda")
        st1.buf_k[:, :, p:] = float("nan")
        lq.lq_la_decode_step(st1, p, q[p:p + 1].cuda(), k[p:p + 1].cuda(), v[p:p + 1].cuda(),
                             alpha.cuda() if heads else alpha[p:p + 1].cuda(), o1)
        assert torch.equal(o1[0], o[p]) and torch.equal(st1.buf_k[0, :, p].cpu(), k[p].float())


def test_decode_forget():
    """alpha = 0: the output is <q, k> v, whatever the state and the window hold."""
    dims, st, *_ = make_state(3, 2, 2, 128, 16, 4, "f32")
    q, k, v, alpha, _ = tokens(4, (2, 2), 128, "f32")
    o = torch.zeros((2, 2, 128), device="cuda")
    one_token(st, [5, 0], q, k, v, torch.zeros_like(alpha), o)
    want = (q.double() * k.double()).sum(-1, keepdim=True) * v.double()
    near(o, want, 2 * R.c_of(128) * (q.abs() * k.abs()).sum(-1, keepdim=True).double() * v.abs().double(), "o")


# ---------------------------------------------------------------------------
# drafted trees
# ---------------------------------------------------------------------------

SHAPES = {
    "chain": lambda n: n - 1,
    "star": lambda n: -1,
    "binary": lambda n: (n - 1) // 2 if n else -1,
    "two chains": lambda n: n - 2 if n >= 2 else -1,
    "mixed": lambda n: -1 if n in (0, 9, 30) else n - 1 if n % 3 else max(0, n - 5),
}


def run_tree(st, pos, parent, q, k, v, alpha, beta, stream=None):
    """beta None: plain linear attention.  Outputs start as MARK."""
    N, B, H, d = q.shape
    gd = st.buf_g.shape[-1]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    full = lambda *s, dt=torch.float32: torch.full(s, MARK, dtype=dt, device="cuda")
    o, tm, tg = full(N, B, H, d, dt=q.dtype), full(B, H, N, d), full(B, H, N, gd)
    args = [x.cuda() for x in (q, k, v, alpha)]
    if beta is None:
        lq.lq_la_tree_step(st, i32(pos), i32(parent), *args, o, tm, tg)
    else:
        lq.lq_gdn_tree_step(st, i32(pos), i32(parent), *args, beta.cuda(), o, tm, tg)
    torch.cuda.synchronize()
    return o, tm, tg


def check_tree(got, hb, bk, bm, bg, pos, parent, q, k, v, alpha, beta):
    o, tm, tg = (x.cpu() for x in got)
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, q, k, v, alpha, beta)
    hn = here.t()                                                           # [N,B]
    near(o[hn], ro[hn], eo[hn], "o", q.dtype)
    on = here[:, None, :, None]
    pick = lambda x: x[on.expand_as(x)]
    # v of bf16 or fp32 is exact in tree_m without the delta rule
    near(pick(tm), pick(rm), pick(em), "tree_m")
    # a log decay: a sum of at most 64 + W logarithms, each off by 2^-22 of itself or of 1
    near(pick(tg), pick(rg), 100 * 2.0 ** -23 * (pick(rg).abs() + 0.05), "tree_g")
    mark = torch.tensor(MARK, dtype=q.dtype).float()
    assert bool((o[~hn].float() == mark).all()) and bool((pick2(tm, ~on) == MARK).all()) and bool((pick2(tg, ~on) == MARK).all())


def pick2(x, m):
    return x[m.expand_as(x)]


@pytest.mark.parametrize("rule", ["gdn", "kda", "la"])
@pytest.mark.parametrize("shape,N", [("chain", 1), ("chain", 5), ("mixed", 16), ("star", 17), ("binary", 31),
                                     ("two chains", 32), ("mixed", 33), ("mixed", 64), ("chain", 64), ("star", 48)])
@pytest.mark.parametrize("d,W,C,io", [(128, 16, 4, "bf16"), (128, 32, 8, "f32"), (64, 16, 3, "f32"), (64, 32, 0, "bf16"),
                                      (16, 4, 1, "f32"), (16, 32, 8, "bf16"), (128, 5, 0, "f32")])
def test_tree_step(rule, shape, N, d, W, C, io):
    pos = [0, W, W // 2, 1, -1, W + 1]
    B, H = len(pos), 2
    per_key = rule == "kda"
    dims, st, hb, bk, bm, bg = make_state(N + d, B, H, d, W, C, io, per_key, slots=[max(p, 0) for p in pos])
    q, k, v, alpha, beta = tokens(N * 7 + W, (N, B, H), d, io, per_key, heads=H if rule == "la" and N % 2 else None)
    alpha = alpha.clamp(min=0.6)
    parent = [[SHAPES[shape](n) for n in range(N)] for _ in range(B)]
    if N > 2:                                        # a row with fewer nodes, a row with invalid entries
        parent[2][N - 1] = -2
        parent[3][N // 2] = N // 2                   # itself: absent, and with it its descendants
        parent[3][1] = 1000000
    before = {f: getattr(st, f).clone() for f in ("sq", "buf_k", "buf_m", "buf_g")}
    got = run_tree(st, pos, parent, q, k, v, alpha, None if rule == "la" else beta)
    check_tree(got, hb, bk, bm, bg, pos, parent, q, k, v, alpha, None if rule == "la" else beta)
    for f, x in before.items():
        assert torch.equal(getattr(st, f).nan_to_num(7.0) if x.is_floating_point() else getattr(st, f),
                           x.nan_to_num(7.0) if x.is_floating_point() else x), f


@pytest.mark.parametrize("rule", ["gdn", "kda", "la"])
@pytest.mark.parametrize("d", [128, 16])
def test_tree_nonfinite_nodes_reach_their_descendants_only(rule, d):
    N, W = 40, 16
    pos, per_key = [3], rule == "kda"
    dims, st, hb, bk, bm, bg = make_state(d, 1, 2, d, W, 2, "f32", per_key, slots=pos)
    q, k, v, alpha, beta = tokens(d, (N, 1, 2), d, "f32", per_key)
    parent = [[SHAPES["two chains"](n) for n in range(N)]]
    parent[0][7] = -2
    clean = [x.clone() for x in (q, k, v)]
    for x in (q, k, v, alpha, beta):                 # an absent node's tokens are not used
        x[7] = float("nan")
    v[20, 0, 0, 3] = float("inf")                    # even chain
    k[25, 0, 1, 2] = float("nan")                    # odd chain after 25: 27, 29, ...
    got = run_tree(st, pos, parent, q, k, v, alpha, None if rule == "la" else beta)
    for x in (alpha, beta):
        x[7] = 1.0
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, *clean, alpha, None if rule == "la" else beta)
    o, tm = got[0].cpu(), got[1].cpu()
    for n in range(N):
        if not here[0, n]:
            continue
        if not (n >= 20 and n % 2 == 0):             # head 0: nodes off the even chain's end
            near(o[n, 0, 0], ro[n, 0, 0], eo[n, 0, 0], f"o {n}")
            near(tm[0, 0, n], rm[0, 0, n], em[0, 0, n], f"m {n}")
        else:
            assert not torch.isfinite(o[n, 0, 0, 3])
        if not (n >= 25 and n % 2):
            near(o[n, 0, 1], ro[n, 0, 1], eo[n, 0, 1], f"o {n}")
            near(tm[0, 1, n], rm[0, 1, n], em[0, 1, n], f"m {n}")
        elif rule != "la":
            assert torch.isnan(o[n, 0, 1]).all()


@pytest.mark.parametrize("d", [128, 64, 16])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_tree_linear_forget(d, io):
    """alpha = 0 at a node: it and its descendants see nothing before it; strong decays do not overflow."""
    N, W, pos = 36, 16, [5, 16]
    dims, st, hb, bk, bm, bg = make_state(d + 1, 2, 2, d, W, 4, io, slots=pos)
    q, k, v, alpha, _ = tokens(d + 2, (N, 2, 2), d, io)
    parent = [[SHAPES["two chains"](n) for n in range(N)], [SHAPES["mixed"](n) for n in range(N)]]
    alpha[6, 0], alpha[13, 0], alpha[20:24, 1] = 0.0, 0.0, 0.0
    alpha[9, 0, 0], alpha[3, 1] = 1e-38, 1e-30
    got = run_tree(st, pos, parent, q, k, v, alpha, None)
    o, tm, tg = (x.cpu() for x in got)
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, q, k, v, alpha)
    near(o, ro, eo, "o", q.dtype)
    assert torch.equal(tm, v.float().permute(1, 2, 0, 3))
    near(tg, rg, 100 * 2.0 ** -23 * (rg.abs() + 0.05), "tree_g")


@pytest.mark.parametrize("rule", ["gdn", "kda"])
@pytest.mark.parametrize("d,io", [(128, "f32"), (128, "bf16"), (64, "f32"), (16, "f32")])
def test_tree_strong_decays(rule, d, io):
    """Decays down to e^-12 a token: exponentials between nodes that are not on one path do not reach a result."""
    N, W, pos = 64, 16, [0, 7, 16]
    per_key = rule == "kda"
    dims, st, hb, bk, bm, bg = make_state(d + 3, 3, 2, d, W, 4, io, per_key, slots=pos)
    q, k, v, alpha, beta = tokens(d + 4, (N, 3, 2), d, io, per_key)
    alpha = torch.exp(-12 * ((alpha - 0.3) / 0.7) ** 4)
    parent = [[SHAPES[x](n) for n in range(N)] for x in ("chain", "mixed", "star")]
    o, tm, tg = (x.cpu() for x in run_tree(st, pos, parent, q, k, v, alpha, beta))
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, q, k, v, alpha, beta)
    # log decays are sums in fp32: at most 8 roundings of |g| on either side of a difference, each a
    # relative error of its exponential, on top of the bounds' c per term
    more = 1 + 16 * float(rg.abs().max()) * R.U / R.c_of(d)
    near(o, ro, more * eo, "o", q.dtype)
    near(tm, rm, more * em, "tree_m")
    near(tg, rg, 100 * 2.0 ** -23 * (rg.abs() + 0.05), "tree_g")


def test_tree_in_a_graph_with_other_trees():
    """A captured tree step replayed with other positions, parents and path lengths (all on the device)."""
    d, W, B, H, N = 128, 16, 3, 2, 33
    dims, st, hb, bk, bm, bg = make_state(40, B, H, d, W, 4, "bf16")
    q, k, v, alpha, beta = tokens(41, (N, B, H), d, "bf16")
    dev = [x.cuda() for x in (q, k, v, alpha, beta)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    full = lambda *s, dt=torch.float32: torch.full(s, MARK, dtype=dt, device="cuda")
    o, tm, tg = full(N, B, H, d, dt=torch.bfloat16), full(B, H, N, d), full(B, H, N, 1)
    pos, parent = i32([0] * B), i32([[-1] * N] * B)
    call = lambda: lq.lq_gdn_tree_step(st, pos, parent, *dev, o, tm, tg)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new_pos, shape in (([16, 0, 7], "chain"), ([1, 17, 15], "mixed"), ([-1, 3, 16], "binary")):
        par = [[SHAPES[shape](n) for n in range(N)] for _ in range(B)]
        par[1][4] = -3
        pos.copy_(i32(new_pos)), parent.copy_(i32(par))
        for x in (o, tm, tg):
            x.fill_(MARK)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_tree((o, tm, tg), hb, bk, bm, bg, new_pos, par, q, k, v, alpha, beta)


@pytest.mark.parametrize("rule,io", [("gdn", "f32"), ("gdn", "bf16"), ("kda", "f32"), ("la", "bf16")])
def test_tree_chain_is_the_decode_steps(rule, io):
    """A chain of drafted tokens gives the decode steps' outputs and window slots (to rounding), and
    the commit of its nodes leaves exactly the nodes' slots."""
    d, W, B, H, N, p0 = 128, 16, 2, 3, 6, 4
    per_key = rule == "kda"
    dims, st, hb, bk, bm, bg = make_state(9, B, H, d, W, 4, io, per_key, slots=[p0] * B)
    dims2, st2, *_ = make_state(9, B, H, d, W, 4, io, per_key, slots=[p0] * B)
    q, k, v, alpha, beta = tokens(10, (N, B, H), d, io, per_key)
    parent = [[n - 1 for n in range(N)]] * B
    o, tm, tg = run_tree(st, [p0] * B, parent, q, k, v, alpha, None if rule == "la" else beta)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    path = i32([list(range(N))] * B)
    lq.lq_tree_commit(st, i32([p0] * B), path, i32([N, 2]), k.cuda(), tm, tg)
    torch.cuda.synchronize()
    assert torch.equal(st.buf_m[0, :, p0:p0 + N], tm[0]) and torch.equal(st.buf_g[0, :, p0:p0 + N], tg[0])
    assert torch.equal(st.buf_k[0, :, p0:p0 + N].cpu(), k[:, 0].transpose(0, 1).float())
    assert torch.equal(st.buf_m[1, :, p0:p0 + 2], tm[1, :, :2]) and torch.isnan(st.buf_m[1, :, p0 + 2:]).all()
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, [p0] * B, parent, q, k, v, alpha, None if rule == "la" else beta)
    od = torch.zeros((B, H, d), dtype=IO[io][1], device="cuda")
    for n in range(N):
        args = [x[n].cuda() for x in (q, k, v, alpha)]
        if rule == "la":
            lq.lq_la_decode_step(st2, p0 + n, *args, od)
        else:
            lq.lq_gdn_decode_step(st2, p0 + n, *args, beta[n].cuda(), od)
        # both are within their bound of the same reference
        near(o[n], ro[n], eo[n], "tree o", IO[io][1])
        near(od, ro[n], 2 * eo[n], "decode o", IO[io][1])
        near(st2.buf_m[:, :, p0 + n], rm[:, :, n], 2 * em[:, :, n], "decode m")


def test_commit_refuses_rows():
    """Rows whose position, count or path is out of range are left untouched; the others are committed."""
    d, W, N, P = 16, 8, 6, 4
    pos = [0, 8, -1, 6, 2, 2, 2, 2, 5]
    n_path = [4, 1, 1, 3, 0, 5, 2, -1, 3]
    path = [[0, 2, 4, 5]] * 6 + [[1, 6, 0, 0], [0, 1, 2, 3], [5, 5, 0, -9]]
    good = [0, 8]
    B = len(pos)
    dims, st, hb, bk, bm, bg = make_state(1, B, 2, d, W, 1, "f32")
    q, k, v, alpha, beta = tokens(2, (N, B, 2), d, "f32")
    o, tm, tg = run_tree(st, [0] * B, [[-1] * N] * B, q, k, v, alpha, beta)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    lq.lq_tree_commit(st, i32(pos), i32(path), i32(n_path), k.cuda(), tm, tg)
    torch.cuda.synchronize()
    want = {"buf_k": bk.clone(), "buf_m": bm.clone(), "buf_g": bg.clone()}
    for b in good:
        for i in range(n_path[b]):
            n, p = path[b][i], pos[b] + i
            want["buf_k"][b, :, p] = k[n, b]
            want["buf_m"][b, :, p], want["buf_g"][b, :, p] = tm[b, :, n].cpu(), tg[b, :, n].cpu()
    for f, x in want.items():
        assert torch.equal(getattr(st, f).cpu(), x), f


@pytest.mark.parametrize("rule", ["gdn", "kda", "la"])
def test_a_served_sequence(rule):
    """The operators as they are used together: a prompt, drafted trees verified and committed, single
    tokens, the flush at the window's end, against the dense recurrence in 64 bits from the same codec."""
    d, W, C, B, H, T = 64, 8, 2, 2, 2, 50
    per_key = rule == "kda"
    dims = lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if per_key else lq.LQ_DECAY_SCALAR, 1)
    st = lq.LayerState.allocate(dims)
    h = torch.zeros((B, H, d, d), device="cuda")
    q, k, v, alpha, beta = [x.cuda() for x in tokens(1, (T, B, H), d, "f32", per_key)]
    o = torch.zeros((T, B, H, d), device="cuda")
    if rule == "la":
        lq.lq_la_prefill(dims, st, None, h, T, q, k, v, alpha, o)
    else:
        lq.lq_gdn_prefill(dims, st, h, T, q, k, v, alpha, beta, o)
    cd = st.codec()
    t = lambda a: torch.from_numpy(a)
    dense = R.dequantize(t(cd["sq"]), t(cd["r"]), t(cd["s"]), t(cd["idx"]), t(cd["cv"]))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    used = 0
    for rnd, (N, paths) in enumerate([(7, [[0, 2, 4], [1]]), (5, [[0, 1], [0, 2, 4]])]):
        q, k, v, alpha, beta = [x.cuda() for x in tokens(50 + rnd, (N, B, H), d, "f32", per_key)]
        parent = [[-1] * N for _ in range(B)]
        for b, p in enumerate(paths):
            for a, c in zip(p, p[1:]):
                parent[b][c] = a
        tm, tg = torch.zeros((B, H, N, d), device="cuda"), torch.zeros((B, H, N, d if per_key else 1), device="cuda")
        ot = torch.zeros((N, B, H, d), device="cuda")
        if rule == "la":
            lq.lq_la_tree_step(st, pos, i32(parent), q, k, v, alpha, ot, tm, tg)
        else:
            lq.lq_gdn_tree_step(st, pos, i32(parent), q, k, v, alpha, beta, ot, tm, tg)
        P = max(len(p) for p in paths)
        lens = i32([len(p) for p in paths])
        lq.lq_tree_commit(st, pos, i32([p + [-1] * (P - len(p)) for p in paths]), lens, k, tm, tg)
        pos += lens
        for b, p in enumerate(paths):
            for n in p:
                dense[b] = step(dense[b], *(x[n, b].double().cpu() for x in (alpha, k, v, beta)), rule)
                want = (dense[b] * q[n, b].double().cpu()[..., None]).sum(-2)
                assert float((ot[n, b].cpu() - want).abs().max() / want.abs().max()) < 1e-5
    assert pos.tolist() == [5, 4]
    q, k, v, alpha, beta = [x.cuda() for x in tokens(99, (B, H), d, "f32", per_key)]
    od = torch.zeros((B, H, d), device="cuda")
    if rule == "la":
        lq.lq_la_decode_step_ragged(st, pos, q, k, v, alpha, od)
    else:
        lq.lq_gdn_decode_step_ragged(st, pos, q, k, v, alpha, beta, od)
    pos += 1
    h_out = torch.zeros((B, H, d, d), device="cuda")
    lq.lq_gdn_window_flush_ragged(st, pos, h_out)
    torch.cuda.synchronize()
    for b in range(B):
        dense[b] = step(dense[b], *(x[b].double().cpu() for x in (alpha, k, v, beta)), rule)
        want = (dense[b] * q[b].double().cpu()[..., None]).sum(-2)
        assert float((od[b].cpu() - want).abs().max() / want.abs().max()) < 1e-5
        # 1e-5: 7 tokens of at most c(64) = 192 * 2^-24 = 1.1e-5 of absolute sums, whose signs are random
        assert float((h_out[b].cpu() - dense[b]).abs().max() / dense[b].abs().max()) < 1e-5


def step(h, alpha, k, v, beta, rule):
    """One token on a dense state [H,d,d]."""
    h = h * (alpha[..., None] if rule == "kda" else alpha[:, None, None])
    u = v if rule == "la" else beta[:, None] * (v - (h * k[..., None]).sum(-2))
    return h + k[..., None] * u[:, None, :]


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

def test_graph_replays_match_eager():
    """A prompt, a tree step, a commit and a decode step in one captured graph, replayed with new inputs
    and eager work between the replays; every replay equals the eager calls bit for bit."""
    d, W, B, H, N, T = 128, 16, 1, 4, 9, 3000
    dims = lq.make_dims(B, H, d, d, W, 4, lq.LQ_DECAY_SCALAR, 1, lq.LQ_IO_BF16)
    ws = torch.empty(max(16, lq.lq_la_workspace_bytes(dims, T)), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    pos, pos2 = i32([3] * B), i32([5] * B)
    parent, path, n_path = i32([[n - 2 if n > 1 else -1 for n in range(N)]] * B), i32([[0, 2]] * B), i32([2] * B)

    def fresh(seed):
        big = [x.cuda() for x in tokens(seed, (T, B, H), d, "bf16")[:4]]
        tr = [x.cuda() for x in tokens(seed + 1, (N, B, H), d, "bf16")]
        one = [x.cuda() for x in tokens(seed + 2, (B, H), d, "bf16")[:4]]
        return big, tr, one

    def buffers():
        z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
        bf = torch.bfloat16
        return dict(st=lq.LayerState.allocate(dims), h=z(B, H, d, d), o=z(T, B, H, d, dt=bf), to=z(N, B, H, d, dt=bf),
                    tm=z(B, H, N, d), tg=z(B, H, N, 1), od=z(B, H, d, dt=bf))

    def calls(x, r, w):
        big, tr, one = x
        lq.lq_la_prefill(dims, r["st"], None, r["h"], T, *big, r["o"], workspace=w)
        lq.lq_gdn_tree_step(r["st"], pos, parent, *tr, r["to"], r["tm"], r["tg"])
        lq.lq_tree_commit(r["st"], pos, path, n_path, tr[1], r["tm"], r["tg"])
        lq.lq_la_decode_step_ragged(r["st"], pos2, *one, r["od"])

    live, ref, got = fresh(1), buffers(), buffers()
    calls(live, got, ws)                                   # warm, eager
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(live, got, ws)
    ws2 = torch.empty_like(ws)
    for rep in range(3):
        new = fresh(100 * rep + 7)
        for a, b in zip(live, new):
            for x, y in zip(a, b):
                x.copy_(y)
        torch.cuda.synchronize()
        calls(live, ref, ws2)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("h", "o", "to", "tm", "tg", "od"):
            assert torch.equal(ref[name], got[name]), (rep, name)
        for f in ("sq", "row_scale", "buf_k", "buf_m", "buf_g"):
            assert torch.equal(getattr(ref["st"], f), getattr(got["st"], f)), (rep, f)


def test_two_streams_at_once():
    """Prompts on two streams at the same time, each with its own workspace, equal the same calls alone."""
    dims = lq.make_dims(1, 4, 128, 128, 16, 4, lq.LQ_DECAY_SCALAR, 1, lq.LQ_IO_BF16)
    T = 5000
    cs = [prefill_case(s, 1, 4, 128, T, "bf16") for s in (1, 2)]
    alone = [run_prefill(*c, "bf16") for c in cs]
    dev = [[x.cuda() for x in c] for c in cs]
    outs = [(torch.zeros((T, 1, 4, 128), dtype=torch.bfloat16, device="cuda"),
             torch.zeros((1, 4, 128, 128), device="cuda")) for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (q, k, v, alpha, h0), (o, h), s in zip(dev, outs, streams):
            lq.lq_la_prefill(dims, None, h0, h, T, q, k, v, alpha, o, stream=s)
    torch.cuda.synchronize()
    for (o, h), (ro, rh) in zip(outs, alone):
        assert torch.equal(o, ro) and torch.equal(h, rh)


def test_results_do_not_depend_on_the_batch():
    """A row computed alone gives the bits it has in a batch (decode and tree; fixed order of sums)."""
    d, W, B, H, N = 128, 16, 5, 3, 20
    pos = [0, 3, 16, 7, 15]
    dims, st, *_ = make_state(77, B, H, d, W, 4, "bf16", slots=pos)
    q, k, v, alpha, beta = tokens(78, (N, B, H), d, "bf16")
    parent = [[SHAPES["mixed"](n) for n in range(N)]] * B
    o, tm, tg = run_tree(st, pos, parent, q, k, v, alpha, beta)
    again = run_tree(st, pos, parent, q, k, v, alpha, beta)
    for x, y in zip((o, tm, tg), again):
        assert torch.equal(x, y)
    for b in (1, 3):
        cut = lambda x: x[:, b:b + 1].contiguous()
        o1, tm1, tg1 = run_tree(st.rows(b, b + 1), pos[b:b + 1], parent[b:b + 1], cut(q), cut(k), cut(v), cut(alpha),
                                cut(beta))
        assert torch.equal(o1[:, 0], o[:, b]) and torch.equal(tm1[0], tm[b]) and torch.equal(tg1[0], tg[b])
