"""Prompts of the gated delta rule over padded batches on the GPU, against the
64-bit recurrence, at the tolerance that fp32 sums give (serving_reference.py)."""
import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
IO = {"f32": (lq.LQ_IO_F32, torch.float32), "bf16": (lq.LQ_IO_BF16, torch.bfloat16)}
MARK = 12345.0       # what untouched rows hold


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def case(seed, B, H, d, T, io, per_key=False, start=True, decay=3.0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    t = IO[io][1]
    q, k = unit(rnd(T, B, H, d)).to(t), unit(rnd(T, B, H, d)).to(t)
    v = rnd(T, B, H, d).to(t)
    alpha = torch.sigmoid(decay - spread * (rnd(T, B, H, d) if per_key else rnd(T, B, H)))
    beta = torch.rand(T, B, H, generator=g)
    return q, k, v, alpha, beta, (0.3 * rnd(B, H, d, d) if start else None)


def dims(q, alpha, io, W=16, C=4):
    T, B, H, d = q.shape
    return lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if alpha.dim() == 4 else lq.LQ_DECAY_SCALAR, 1, IO[io][0])


def run(q, k, v, alpha, beta, h0, io, lens=None, st=None, with_o=True, stream=None):
    T, B, H, d = q.shape
    dm = dims(q, alpha, io)
    dev = lambda x: None if x is None else x.cuda().contiguous()
    o = torch.full((T, B, H, d), MARK, dtype=IO[io][1], device="cuda") if with_o else None
    h = torch.full((B, H, d, d), MARK, device="cuda")
    need = lq.lq_gdn_workspace_bytes(dm, T)
    w = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") if need else None       # garbage: NaN bits
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    lq.lq_gdn_prefill_ragged(dm, st, dev(h0), h, T, dev(q), dev(k), dev(v), dev(alpha), dev(beta), o, lens=lens,
                             workspace=w)
    torch.cuda.synchronize()
    return o, h


def near(got, ref, d, what, dtype=torch.float32):
    """At most the tolerance of the largest value, and half a step of the output's type."""
    got, ref = got.double().cpu(), ref.cpu()
    lim = R.gdn_tolerance(d) * float(ref.abs().max()) + torch.finfo(dtype).eps / 2 * (dtype != torch.float32) * ref.abs() * 1.01
    worst = float(((got - ref).abs() / (lim + 1e-37)).max())
    assert worst <= 1, f"{what}: {worst:.2f} times the tolerance"


def check(o, h, c, io, lens=None, what=""):
    q, k, v, alpha, beta, h0 = c
    T, d = q.shape[0], q.shape[-1]
    cu = lambda x: None if x is None else x.cuda()
    lt = None if lens is None else torch.tensor(lens).clamp(0, T)
    ro, rh = R.gdn_prefill(cu(q), cu(k), cu(v), cu(alpha), cu(beta), cu(h0), lt)
    near(h, rh, d, what + " h")
    if o is not None:
        real = torch.ones(q.shape[:2], dtype=torch.bool) if lens is None else torch.arange(T)[:, None] < lt[None]
        if real.any():
            near(o.cpu()[real], ro.cpu()[real], d, what + " o", IO[io][1])
        assert bool((o.cpu()[~real].float() == torch.tensor(MARK, dtype=IO[io][1]).float()).all()), "rows past a length"


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 7, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 130])
def test_lengths(T, d, per_key, io):
    c = case(T * 100 + d, 2, 3, d, T, io, per_key, start=T % 3 != 0)
    check(*run(*c, io), c, io)


@pytest.mark.parametrize("B,H,d,T,io,per_key", [
    (1, 1, 128, 1500, "bf16", False), (1, 2, 128, 2049, "f32", False), (3, 1, 64, 1111, "bf16", False),
    (1, 1, 64, 900, "f32", True), (1, 3, 16, 1300, "bf16", False), (2, 1, 16, 777, "f32", True),
    (1, 16, 128, 4096, "bf16", False), (1, 1, 128, 9001, "bf16", False), (1, 2, 128, 1333, "bf16", True),
    (1, 1, 128, 700, "f32", True), (2, 2, 64, 1025, "bf16", True)])
def test_long_prompts_of_few_heads(B, H, d, T, io, per_key):
    c = case(T, B, H, d, T, io, per_key)
    check(*run(*c, io), c, io)


@pytest.mark.parametrize("B,H,d,T,io,per_key", [
    (40, 33, 128, 40, "bf16", False), (10, 13, 128, 200, "f32", False), (13, 10, 128, 300, "bf16", False),
    (129, 1, 64, 150, "f32", False), (64, 2, 64, 150, "bf16", False), (150, 30, 16, 40, "bf16", False),
    (20, 33, 128, 70, "bf16", True), (64, 5, 64, 70, "f32", True)])
def test_many_heads(B, H, d, T, io, per_key):
    c = case(5, B, H, d, T, io, per_key, start=False)
    check(*run(*c, io), c, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d,T", [(128, 70), (64, 70), (16, 70), (128, 1400), (64, 1400), (16, 1400), (128, 3)])
def test_padded_rows(d, T, per_key, io):
    """Tokens past a row's length may hold NaN; their o rows stay; rows without tokens keep h0."""
    q, k, v, alpha, beta, h0 = case(7 * d + T, 7, 2, d, T, io, per_key)
    lens = [T, 0, 1, T - 1, -4, T + 9, T // 2]
    real = torch.arange(T)[:, None] < torch.tensor(lens)[None]
    nan = float("nan")
    q, k, v = (torch.where(real[..., None, None], x, nan).to(x.dtype) for x in (q, k, v))
    alpha = torch.where(real[(...,) + (None,) * (alpha.dim() - 2)], alpha, nan)
    beta = torch.where(real[..., None], beta, nan)
    c = (q, k, v, alpha, beta, h0)
    o, h = run(*c, io, lens=lens)
    assert bool(torch.isfinite(h).all())
    check(o, h, c, io, lens=lens)
    assert torch.equal(h[1].cpu(), h0[1]) and torch.equal(h[4].cpu(), h0[4])


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("T", [0, 3, 40, 1300])
def test_rows_without_tokens_and_without_a_start(T, d):
    q, k, v, alpha, beta, _ = case(T, 2, 2, d, max(T, 1), "bf16", start=False)
    if T == 0:
        h = torch.full((2, 2, d, d), MARK, device="cuda")
        dm = dims(q, alpha, "bf16")
        lq.lq_gdn_prefill_ragged(dm, None, None, h, 0, None, None, None, None, None)
        assert float(h.abs().max()) == 0.0
        h0 = torch.randn(2, 2, d, d, device="cuda")
        lq.lq_gdn_prefill_ragged(dm, None, h0, h, 0, None, None, None, None, None)
        assert torch.equal(h, h0)
        return
    c = (q, k, v, alpha, beta, None)
    o, h = run(*c, "bf16", lens=[0, T])
    check(o, h, c, "bf16", lens=[0, T])
    assert float(h[0].abs().max()) == 0.0


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_strong_decays_and_forgetting(d, per_key, io):
    """Decays from 1 to far below fp32's smallest product within a chunk, and tokens that forget everything."""
    T = 200
    q, k, v, alpha, beta, h0 = case(d, 1, 3, d, T, io, per_key)
    g = torch.Generator().manual_seed(9)
    x = torch.rand(alpha.shape, generator=g)
    alpha = torch.where(x < 0.3, torch.exp(-60 * torch.rand(alpha.shape, generator=g)), alpha)
    alpha = torch.where(x > 0.95, torch.ones_like(alpha), alpha)
    alpha = torch.where((x > 0.4) & (x < 0.44), torch.zeros_like(alpha), alpha)
    alpha[:, 0, 0] = 1.0                                   # no decay at all
    c = (q, k, v, alpha, beta, h0)
    check(*run(*c, io), c, io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_keys_that_repeat(d, per_key, io):
    """One key for every token with full steps (each token replaces the one before), and steps of 0."""
    T = 100
    q, k, v, alpha, beta, h0 = case(d + 1, 1, 2, d, T, io, per_key, decay=6.0)
    k = k[:1].expand_as(k).contiguous()
    beta = torch.ones_like(beta)
    beta[40:45] = 0.0
    c = (q, k, v, alpha, beta, h0)
    check(*run(*c, io), c, io)


@pytest.mark.parametrize("d,T,per_key", [(128, 300, False), (128, 40, True), (16, 300, False), (64, 700, False),
                                         (128, 2, False), (16, 3, True)])
def test_state_without_outputs_in_place_and_codec(d, T, per_key):
    """No outputs: the same state to rounding; h0 may be h; the codec is that of the state written."""
    c = case(3, 2, 3, d, T, "bf16", per_key)
    o, h = run(*c, "bf16")
    _, h1 = run(*c, "bf16", with_o=False)
    near(h1, h.double(), d, "without outputs")
    dm = dims(c[0], c[3], "bf16")
    st, want = lq.LayerState.allocate(dm), lq.LayerState.allocate(dm)
    x = c[5].cuda().clone()
    args = [t.cuda() for t in c[:5]]
    o2 = torch.empty_like(o)
    lq.lq_gdn_prefill_ragged(dm, st, x, x, T, *args, o2)             # the workspace allocated by the call
    assert torch.equal(x, h) and torch.equal(o2, o)
    lq.lq_gdn_state_quantize(want, h)
    for f in ("sq", "row_scale", "col_scale", "comp_idx", "comp_val"):
        assert torch.equal(getattr(st, f), getattr(want, f)), f


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T,per_key,bad", [(128, 150, False, 70), (128, 90, True, 37), (64, 150, False, 64),
                                             (16, 90, False, 20), (64, 60, True, 33), (128, 3, False, 1),
                                             (128, 1500, False, 700), (16, 40, True, 17)])
def test_values_that_are_not_finite_stay_where_they_belong(d, T, per_key, bad, io):
    """A v reaches its own column from its own token on; a k, alpha or beta its head from its token on;
    a q its own output.  Everything before, and every other head, is as without it."""
    q, k, v, alpha, beta, h0 = case(bad, 1, 6, d, T, io, per_key)
    clean = (q, k, v, alpha, beta, h0)
    ro, rh = R.gdn_prefill(*clean)
    q, k, v, alpha, beta = (x.clone() for x in (q, k, v, alpha, beta))
    nan, inf = float("nan"), float("inf")
    v[bad, 0, 0, 5] = nan
    k[bad, 0, 1, 3] = nan
    q[bad, 0, 2, 1] = inf
    beta[bad, 0, 3] = nan
    if per_key:
        alpha[bad, 0, 4, 2] = nan
    else:
        alpha[bad, 0, 4] = nan
    o, h = run(q, k, v, alpha, beta, h0, io)
    o, h, t = o.cpu(), h.cpu(), torch.arange(T)
    ok = torch.ones(T, 6, d, dtype=torch.bool)
    ok[bad:, 0, 5] = False
    for hd in (1, 3):
        ok[bad:, hd] = False
    ok[bad, 2] = False
    ok[bad:, 4] = False
    hk = torch.ones(6, d, d, dtype=torch.bool)
    hk[0, :, 5] = False
    hk[[1, 3, 4]] = False
    assert bool(torch.isfinite(o[:, 0][ok].float()).all()) and bool(torch.isfinite(h[0][hk]).all())
    for hd in range(6):                                    # (a head's own scale)
        m = ok[:, hd]
        near(o[:, 0, hd][m], ro[:, 0, hd][m], d, f"o {hd}", IO[io][1])
        if hk[hd].any():
            near(h[0, hd][hk[hd]], rh[0, hd][hk[hd]], d, f"h {hd}")
    assert not bool(torch.isfinite(o[bad:, 0, 0, 5].float()).any()) and not bool(torch.isfinite(h[0, 0, :, 5]).any())
    assert not bool(torch.isfinite(o[bad:, 0, 1].float()).any()) and not bool(torch.isfinite(h[0, 3]).any())
    assert not bool(torch.isfinite(o[bad, 0, 2].float()).any())


@pytest.mark.parametrize("d,T,io,per_key", [(128, 600, "bf16", False), (128, 33, "f32", True), (16, 900, "f32", False),
                                            (64, 2, "bf16", False)])
def test_calls_repeat_bit_for_bit_on_streams_and_in_graphs(d, T, io, per_key):
    """Another stream, two calls at once with a workspace each, and replays of a captured call with other
    work between them give the bits of the plain call."""
    c = case(8, 2, 4, d, T, io, per_key)
    dm = dims(c[0], c[3], io)
    x = [t.cuda() for t in c]
    o0, h0 = run(*c, io)
    need = lq.lq_gdn_workspace_bytes(dm, T)
    outs = [(torch.zeros_like(o0), torch.zeros_like(h0), torch.empty(need, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, (o, h, w) in zip(streams, outs):
        lq.lq_gdn_prefill_ragged(dm, None, x[5], h, T, *x[:5], o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, h, _ in outs:
        assert torch.equal(o, o0) and torch.equal(h, h0)
    o, h, w = outs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lq.lq_gdn_prefill_ragged(dm, None, x[5], h, T, *x[:5], o, workspace=w)
    for _ in range(3):
        o.zero_()
        h.zero_()
        w.fill_(0xff)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o0) and torch.equal(h, h0)


def test_equals_the_lockstep_prompt_to_rounding():
    """lq_gdn_prefill over the same tokens."""
    for per_key in (False, True):
        q, k, v, alpha, beta, h0 = c = case(2, 2, 3, 128, 100, "f32", per_key)
        o, h = run(*c, "f32")
        dm = dims(q, alpha, "f32")
        h1, o1 = h0.cuda(), torch.empty_like(o)
        lq.lq_gdn_prefill(dm, None, h1, 100, *[t.cuda() for t in c[:5]], o1)
        near(h, h1.double(), 128, "h")
        near(o, o1.double(), 128, "o")


def test_sizes_and_overlaps_are_refused():
    c = case(1, 2, 2, 16, 8, "f32")
    dm = dims(c[0], c[3], "f32")
    q, k, v, alpha, beta, h0 = (t.cuda() for t in c)
    h, o = torch.empty_like(h0), torch.empty_like(q)
    call = lambda h0=h0, h=h, q=q, alpha=alpha, beta=beta, o=o, **kw: lq.lq_gdn_prefill_ragged(
        dm, None, h0, h, 8, q, k, v, alpha, beta, o, **kw)
    call()
    flat = torch.zeros(2 * h.numel(), device="cuda")
    part = flat[64:64 + h.numel()].view(h.shape)
    for kw in (dict(q=q[:7]), dict(alpha=alpha[..., None]), dict(beta=beta.double()), dict(o=o.transpose(1, 2)),
               dict(h0=h0.cpu()), dict(h0=part, h=flat[:h.numel()].view(h.shape)), dict(lens=torch.zeros(3, device="cuda")),
               dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    st = lq.LayerState.allocate(lq.make_dims(2, 3, 16, 16, 16, 4))
    with pytest.raises(ValueError):
        lq.lq_gdn_prefill_ragged(dm, st, h0, h, 8, q, k, v, alpha, beta, o)
