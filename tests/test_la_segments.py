"""Which prompts are cut into segments, as lq_la_workspace_bytes tells (host only)."""
import os

import pytest

from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.skipif(not os.path.exists(lq.LIB_PATH), reason="liblq.so not built")


def need(B, H, d, T, io):
    return lq.lq_la_workspace_bytes(lq.make_dims(B, H, d, d, 16, 4, lq.LQ_DECAY_SCALAR, 1, io), T)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("io,chunk", [(lq.LQ_IO_F32, 32), (lq.LQ_IO_BF16, 64)])
def test_prompts_of_two_chunks_run_in_one_launch(d, io, chunk):
    for B, H in ((1, 1), (1, 16), (4, 32)):
        for T in (chunk, chunk + 1, 2 * chunk):
            assert need(B, H, d, T, io) == 0
        assert need(B, H, d, 2 * chunk + 1, io) > 0
        sizes = [need(B, H, d, T, io) for T in range(1, 12 * chunk, 7)]
        assert sizes == sorted(sizes)
