"""What the bits of a row of linear attention depend on, across batches."""
import pytest
import torch

import la_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
IO = {"f32": (lq.LQ_IO_F32, torch.float32), "bf16": (lq.LQ_IO_BF16, torch.bfloat16)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def tokens(seed, T, B, H, d, io):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, device="cuda", generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    t = IO[io][1]
    alpha = torch.sigmoid(3.0 - rn(T, B, H))
    return unit(rn(T, B, H, d)).to(t), unit(rn(T, B, H, d)).to(t), rn(T, B, H, d).to(t), alpha


def prefill(q, k, v, alpha, io, h0=None, lens=None):
    T, B, H, d = q.shape
    dims = lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    o, h = torch.zeros((T, B, H, d), dtype=IO[io][1], device="cuda"), torch.zeros((B, H, d, d), device="cuda")
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    lq.lq_la_prefill(dims, None, h0, h, T, q, k, v, alpha, o, lens=lens)
    torch.cuda.synchronize()
    return o, h


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 64])
def test_prompts_of_more_than_131072_heads(d, io):
    """They run by chunks as smaller batches do (d = 64: up to 262144 heads, d = 16: any number): the last rows
    have the bits that they have by themselves, and the values of the definition."""
    B, H, T, b0 = 1025, 128, 9, 1000
    x = tokens(d, T, B, H, d, io)
    o, h = prefill(*x, io)
    cut = [y[:, b0:].contiguous() for y in x]
    o1, h1 = prefill(*cut, io)
    assert torch.equal(o[:, b0:], o1) and torch.equal(h[b0:], h1)
    few = [y[:, -1:].contiguous() for y in x]
    ro, rh, oa, ha = R.la_prefill(*few)
    c = R.c_of(d) + 4 * R.U
    assert bool(((h[-1:].double() - rh).abs() <= c * ha).all())
    lim = c * oa + R.half_step(IO[io][1]) * (ro.abs() + c * oa) + 1e-37
    assert bool(((o[:, -1:].double() - ro).abs() <= lim).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(16, 600), (64, 600), (128, 600), (128, 3), (128, 40)])
def test_a_row_does_not_depend_on_what_the_others_hold(d, T, io):
    """The same B, H and T (prompts in segments, whole and token by token): other tokens, lengths, states and
    infinities in the other rows leave a row's bits."""
    B, H, keep = 4, 2, 2
    x, y = tokens(1, T, B, H, d, io), tokens(2, T, B, H, d, io)
    h0, h0b = torch.randn(B, H, d, d, device="cuda"), torch.randn(B, H, d, d, device="cuda")
    for a, b in zip((*x, ), y):
        b[:, keep] = a[:, keep]
    h0b[keep] = h0[keep]
    y[2][T // 2, 0] = float("inf")
    y[1][0, 1] = float("nan")
    o, h = prefill(*x, io, h0, [T, T, T - 1, T])
    o1, h1 = prefill(*y, io, h0b, [T, T // 2, T - 1, 0])
    assert torch.equal(o[:, keep], o1[:, keep]) and torch.equal(h[keep], h1[keep])
    o2, h2 = prefill(*x, io, h0, [T, T, T - 1, T])
    assert torch.equal(o, o2) and torch.equal(h, h2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,B,H,T", [(128, 6, 40, 150), (64, 8, 40, 150), (16, 21, 40, 150), (128, 3, 2, 31),
                                     (64, 3, 2, 31), (16, 3, 2, 100)])
def test_prompts_without_a_workspace_have_the_same_bits_in_every_batch(d, B, H, T, io):
    """Part of a batch and a longer padding, as long as neither call needs a workspace."""
    part, pad = B - 1, 40 if T == 150 else 1
    flag = IO[io][0]
    for b, t in ((B, T), (part, T), (B, T + pad)):
        assert lq.lq_la_workspace_bytes(lq.make_dims(b, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, flag), t) == 0
    x = tokens(3, T, B, H, d, io)
    h0 = torch.randn(B, H, d, d, device="cuda")
    o, h = prefill(*x, io, h0)
    o1, h1 = prefill(*(y[:, :part].contiguous() for y in x), io, h0[:part])
    assert torch.equal(o[:, :part], o1) and torch.equal(h[:part], h1)
    longer = [torch.cat([y, torch.full_like(y[:1].expand(pad, *y.shape[1:]), float("nan"))]) for y in x]
    o2, h2 = prefill(*longer, io, h0, [T] * B)
    assert torch.equal(o, o2[:T]) and torch.equal(h, h2) and float(o2[T:].float().abs().max()) == 0.0


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompts_in_segments_agree_to_rounding_in_every_batch(io):
    """A row of a batch of 1, 4 and 5 rows of 32 heads (16, 4 and one segment at most), each within the bounds
    of the definition."""
    T, H, d = 700, 32, 128
    x = tokens(4, T, 5, H, d, io)
    row = [y[:, :1].contiguous() for y in x]
    ro, rh, oa, ha = R.la_prefill(*row)
    c = R.c_of(d) + 2 * (T / 16 + 1) * R.U
    sizes = set()
    for b in (1, 4, 5):
        sizes.add(lq.lq_la_workspace_bytes(lq.make_dims(b, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0]), T) // b)
        o, h = prefill(*(y[:, :b].contiguous() for y in x), io)
        assert bool(((h[:1].double() - rh).abs() <= c * ha).all())
        assert bool(((o[:, :1].double() - ro).abs() <= c * oa + R.half_step(IO[io][1]) * (ro.abs() + c * oa) + 1e-37).all())
    assert len(sizes) == 3                                # three different cuts


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_a_decoded_row_has_the_same_bits_in_every_batch(d, io):
    """Ragged and lockstep, in a batch and alone."""
    B, H, W, p = 5, 3, 16, 9
    dims = lq.make_dims(B, H, d, d, W, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0])
    st = lq.LayerState.allocate(dims)
    g = torch.Generator(device="cuda").manual_seed(d)
    lq.lq_gdn_state_quantize(st, torch.randn(B, H, d, d, device="cuda", generator=g))
    for f in (st.buf_k, st.buf_m):
        f.normal_(generator=g)
    st.buf_g.copy_(-0.1 * torch.rand(B, H, W, 1, device="cuda", generator=g).cumsum(2))
    q, k, v, alpha = (y[0] for y in tokens(5, 1, B, H, d, io))
    kept = [f.clone() for f in (st.buf_k, st.buf_m, st.buf_g)]
    pos = torch.tensor([0, 3, p, 15, 7], dtype=torch.int32, device="cuda")
    o = torch.zeros((B, H, d), dtype=IO[io][1], device="cuda")
    lq.lq_la_decode_step_ragged(st, pos, q, k, v, alpha, o)
    for b in range(B):
        for f, was in zip((st.buf_k, st.buf_m, st.buf_g), kept):
            f.copy_(was)
        one = lq.LayerState(lq.make_dims(1, H, d, d, W, 4, lq.LQ_DECAY_SCALAR, 1, IO[io][0]),
                            *(getattr(st, n)[b:b + 1].clone() for n in lq._STATE_FIELDS))
        args = [y[b:b + 1].contiguous() for y in (q, k, v, alpha)]
        o1, o2 = torch.zeros_like(o[:1]), torch.zeros_like(o[:1])
        lq.lq_la_decode_step_ragged(one, pos[b:b + 1].contiguous(), *args, o1)
        g1 = one.buf_g.clone()
        lq.lq_la_decode_step(one, int(pos[b]), *args, o2)
        assert torch.equal(o1[0], o[b]) and torch.equal(o2[0], o[b]) and torch.equal(g1, one.buf_g)
