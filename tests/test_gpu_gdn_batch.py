"""What the bits of a row of gated-delta-rule prompts depend on, across batches."""
import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
IO = {"f32": (lq.LQ_IO_F32, torch.float32), "bf16": (lq.LQ_IO_BF16, torch.bfloat16)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def tokens(seed, T, B, H, d, io, per_key):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, device="cuda", generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    t = IO[io][1]
    alpha = torch.sigmoid(3.0 - (rn(T, B, H, d) if per_key else rn(T, B, H)))
    return unit(rn(T, B, H, d)).to(t), unit(rn(T, B, H, d)).to(t), rn(T, B, H, d).to(t), alpha, torch.sigmoid(rn(T, B, H))


def shape(B, H, d, io, per_key):
    return lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_PER_KEY if per_key else lq.LQ_DECAY_SCALAR, 1, IO[io][0])


def prompt(x, io, h0=None, lens=None):
    T, B, H, d = x[0].shape
    dims = shape(B, H, d, io, x[3].dim() == 4)
    o, h = torch.zeros((T, B, H, d), dtype=IO[io][1], device="cuda"), torch.zeros((B, H, d, d), device="cuda")
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    lq.lq_gdn_prefill_ragged(dims, None, h0, h, T, *x, o, lens=lens)
    torch.cuda.synchronize()
    return o, h


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d,T", [(16, 600), (64, 600), (128, 600), (128, 3), (128, 40), (64, 70)])
def test_a_row_does_not_depend_on_what_the_others_hold(d, T, per_key, io):
    """The same B, H and T (prompts in segments, whole and token by token): other tokens, lengths, decays,
    states, infinities and NaN in the other rows leave a row's bits; and a call gives its bits again."""
    B, H, keep = 4, 2, 2
    x, y = tokens(1, T, B, H, d, io, per_key), tokens(2, T, B, H, d, io, per_key)
    h0, h0b = torch.randn(B, H, d, d, device="cuda"), torch.randn(B, H, d, d, device="cuda")
    for a, b in zip(x, y):
        b[:, keep] = a[:, keep]
    h0b[keep] = h0[keep]
    y[2][T // 2, 0] = float("inf")
    y[1][0, 1] = float("nan")
    y[3][:, 3] = 0.0
    o, h = prompt(x, io, h0, [T, T, T - 1, T])
    o1, h1 = prompt(y, io, h0b, [T, T // 2, T - 1, T])
    assert torch.equal(o[:, keep], o1[:, keep]) and torch.equal(h[keep], h1[keep])
    o2, h2 = prompt(x, io, h0, [T, T, T - 1, T])
    assert torch.equal(o, o2) and torch.equal(h, h2)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d,B,H,T", [(128, 5, 40, 230), (64, 8, 40, 230), (16, 15, 40, 230), (128, 3, 2, 150),
                                     (64, 3, 2, 31), (16, 3, 2, 100)])
def test_prompts_without_a_workspace_have_the_same_bits_in_every_batch(d, B, H, T, per_key, io):
    """Part of a batch and a longer padding, as long as neither call needs a workspace."""
    part, pad = B - 1, 40
    for b, t in ((B, T), (part, T), (B, T + pad)):
        assert lq.lq_gdn_workspace_bytes(shape(b, H, d, io, per_key), t) == 0
    x = tokens(3, T, B, H, d, io, per_key)
    h0 = torch.randn(B, H, d, d, device="cuda")
    o, h = prompt(x, io, h0)
    o1, h1 = prompt([y[:, :part].contiguous() for y in x], io, h0[:part])
    assert torch.equal(o[:, :part], o1) and torch.equal(h[:part], h1)
    longer = [torch.cat([y, torch.full_like(y[:1].expand(pad, *y.shape[1:]), float("nan"))]) for y in x]
    o2, h2 = prompt(longer, io, h0, [T] * B)
    assert torch.equal(o, o2[:T]) and torch.equal(h, h2) and float(o2[T:].float().abs().max()) == 0.0


@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_prompts_of_more_than_131072_heads(d, per_key):
    """By chunks up to 2^24 / d heads (d = 16: any number), by the recurrence beyond: the last rows against
    the definition, and, where both run by chunks, the bits that they have in a small batch."""
    B, H, T, io = 1025, 128, 9, "bf16"
    x = tokens(d, T, B, H, d, io, per_key)
    o, h = prompt(x, io)
    cut = [y[:, -2:].contiguous() for y in x]
    ro, rh = R.gdn_prefill(*cut)
    tol = R.gdn_tolerance(d)
    assert float((h[-2:].double() - rh).abs().max()) <= tol * float(rh.abs().max())
    lim = tol * float(ro.abs().max()) + torch.finfo(torch.bfloat16).eps / 2 * ro.abs() * 1.01
    assert bool(((o[:, -2:].double() - ro).abs() <= lim).all())
    if d < 128:
        o1, h1 = prompt(cut, io)
        assert torch.equal(o[:, -2:], o1) and torch.equal(h[-2:], h1)
