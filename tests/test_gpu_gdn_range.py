"""Prompts with a decay per key channel, strong decays and values far from 1, against the 64-bit
recurrence at the tolerance that fp32 sums give."""
import pytest
import torch

from recurrent_state_quant_lq_amd import lq
from test_gpu_gdn_prompt import case, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("size", [1e13, 2.0 ** 60, 1e-20])
@pytest.mark.parametrize("steps", [0.5, 2.75, 3.0, 5.5, 11.5])
def test_strong_decays(steps, size, d, io):
    """Channels that lose 2^-steps a token (and others that keep): chunks of 32 (d = 16: of 16) tokens
    up to those where a channel's product comes next to the border of a chunk."""
    T = 70
    q, k, v, alpha, beta, h0 = case(int(4 * steps) + d, 2, 2, d, T, io, True)
    far = torch.arange(d) % 3 == 1
    alpha = torch.where(far, 2.0 ** -steps * (1.0 - 1e-3 * torch.rand(alpha.shape)), alpha)
    c = (q, k, (v.float() * size).to(v.dtype), alpha, beta, h0 * size)
    o, h = run(*c, io)
    assert bool(torch.isfinite(h).all()) and bool(torch.isfinite(o).all())
    check(o, h, c, io)
