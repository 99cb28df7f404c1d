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
