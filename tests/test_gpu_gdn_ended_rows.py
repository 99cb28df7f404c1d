"""Prompts of few heads, cut into segments: rows that end before later segments keep what they hold, bit for bit."""
import pytest
import torch

from recurrent_state_quant_lq_amd import lq
from test_gpu_gdn_prompt import IO, case, dims

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def call(c, io, lens, with_o, in_place=False):
    q, k, v, alpha, beta, h0 = c
    T, B, H, d = q.shape
    dm = dims(q, alpha, io)
    dev = [x.cuda() for x in (q, k, v, alpha, beta)]
    o = torch.zeros(T, B, H, d, dtype=IO[io][1], device="cuda") if with_o else None
    start = h0.cuda()
    h = start if in_place else torch.full_like(start, 7.0)
    lq.lq_gdn_prefill_ragged(dm, None, start, h, T, *dev, o, lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    return o, h.cpu()


bits = lambda x: x.contiguous().view(torch.int32)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("with_o,in_place", [(True, False), (False, False), (True, True)])
def test_ended_rows_keep_their_bits(d, per_key, io, with_o, in_place):
    """Row 0 has no tokens and a state with infinities, NaN, zeros of both signs and values next to
    zero: h is h0.  Row 1 ends in the first segment, with an infinity in one value column: h is that
    of a call of its length, whose one segment computes it in the same order."""
    T, n = 700, 40
    q, k, v, alpha, beta, h0 = case(3 * d, 3, 2, d, T, io, per_key)
    h0[0, 0, 1, 2], h0[0, 0, 3, 5], h0[0, 1, 4, 4] = float("inf"), float("nan"), float("-inf")
    h0[0, :, 6] = torch.where(torch.arange(d) % 2 == 0, 0.0, -0.0)
    h0[0, :, 7] = torch.randn(2, d) * 1e-38
    h0[0, :, 8] = torch.randn(2, d) * 1e-41
    h0[1, :, 9] = torch.randn(2, d) * 1e-37
    v[n - 1, 1, :, 3] = float("inf")
    c = (q, k, v, alpha, beta, h0)
    assert lq.lq_gdn_workspace_bytes(dims(q, alpha, io), T) > 0 == lq.lq_gdn_workspace_bytes(dims(q, alpha, io), n)
    _, h = call(c, io, [0, n, T], with_o, in_place)
    assert torch.equal(bits(h[0]), bits(h0[0]))
    short = tuple(x[:n].contiguous() for x in c[:5]) + (h0,)
    _, want = call(short, io, [n] * 3, with_o)
    other = torch.arange(d) != 3
    assert not torch.isfinite(want[1, :, :, 3]).any() and torch.isfinite(want[1][:, :, other]).all()
    assert torch.equal(bits(h[1][:, :, other]), bits(want[1][:, :, other]))
    assert not torch.isfinite(h[1, :, :, 3]).any()
