"""Host-only checks: overlapping arrays are refused before any HIP call."""
import ctypes as ct
import os
import random

import pytest

from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.skipif(not os.path.exists(lq.LIB_PATH), reason="liblq.so not built")

A = ct.c_void_p(0x7000000)      # an aligned address that is never dereferenced
NAMES = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")


def _dims(**kw):
    base = dict(B=2, H=3, dk=128, dv=128, W=16, C=4, decay_mode=0, smooth=1, io_dtype=0)
    base.update(kw)
    return lq.lq_dims(*[base[n] for n in ("B", "H", "dk", "dv", "W", "C", "decay_mode", "smooth", "io_dtype")])


def _bytes(d, rows):
    g = d.dk if d.decay_mode else 1
    return [rows * d.H * x for x in (d.dk * d.dk, d.dk * 4, d.dk * 4, d.C * 4, d.C * d.dk * 4, d.W * d.dk * 4,
                                     d.W * d.dk * 4, d.W * g * 4)]


def _gather(d, dst, src, rows, pos=A, pos_out=None):
    pk = lambda x: (lq.lq_state * len(x))(*[lq.lq_state(*s) for s in x])
    return lq.load().lq_state_gather(ct.byref(d), len(dst), pk(dst), pk(src), rows, A, pos, pos_out, None)


def _layout(d, rows_of, rng):
    """States of rows_of[i] rows side by side in a random order, and the next free address."""
    parts = [(i, f) for i in range(len(rows_of)) for f in range(8)]
    rng.shuffle(parts)
    at, states = 0x10000000, [[0] * 8 for _ in rows_of]
    for i, f in parts:
        states[i][f] = at
        at += _bytes(d, rows_of[i])[f] + 15 & ~15
    return states, at


@pytest.mark.parametrize("layers", [1, 2, 5, 40])
@pytest.mark.parametrize("per_key", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_every_written_array_against_all_others(layers, per_key, in_place):
    """Arrays packed side by side; then one of them is moved onto another one's first or last bytes.  What is accepted
    is shown by the end of the checks: positions that would be written over the index are refused last."""
    rng = random.Random(layers + 100 * per_key)
    d, rows = _dims(decay_mode=per_key), 2 if in_place else 3
    last = ct.c_void_p(0x6000000)
    for _ in range(30):
        states, free = _layout(d, [d.B] * layers + ([] if in_place else [rows] * layers), rng)
        dst, src = states[:layers], states[:layers] if in_place else states[layers:]
        src = [list(x) for x in src]
        # the whole layout stands: only the written positions collide (with the last array's last word)
        ends = [(s[f] + _bytes(d, r)[f], s[f]) for s, r in [(x, d.B) for x in dst] + [(x, rows) for x in src] for f in range(8)]
        assert _gather(d, dst, src, rows, pos=last, pos_out=ct.c_void_p(max(ends)[0] - 4)) == lq.LQ_ERR_OVERLAP
        l, f, m, g = rng.randrange(layers), rng.randrange(8), rng.randrange(layers), rng.randrange(8)
        to_src = not in_place and rng.random() < 0.5
        if not to_src and (l, f) == (m, g):
            continue
        over, size = ((src[m][g], _bytes(d, rows)[g]) if to_src else (dst[m][g], _bytes(d, d.B)[g]))
        mine = _bytes(d, d.B)[f]
        at = rng.choice([over, over + size - 16 & ~15, max(over - mine + 16, 0x1000) & ~15])
        dst[l][f] = at
        if in_place:
            src[l][f] = at
        assert _gather(d, dst, src, rows, pos=last) == lq.LQ_ERR_OVERLAP, (l, f, m, g, to_src)


def test_fields_that_are_not_the_same():
    """A row scale inside another layer's compensators, inside its own layer's, a window over a codec."""
    d = _dims()
    base = lambda i: [0x10000000 * i + 0x1000000 * f for f in range(8)]
    dst, src = [base(1), base(2)], [base(3), base(4)]
    for l, f, at in ((0, 1, base(2)[4]), (0, 1, base(1)[4]), (1, 5, base(1)[0]), (1, 6, base(3)[2]), (0, 7, base(4)[7])):
        x = [list(s) for s in dst]
        x[l][f] = at
        assert _gather(d, x, src, 2) == lq.LQ_ERR_OVERLAP
    # windows do not count without positions
    x = [list(s) for s in dst]
    x[0][5] = x[1][5] = x[0][0]
    assert _gather(d, x, src, 2, pos=None, pos_out=A) == lq.LQ_ERR_OVERLAP      # (the index)


@pytest.mark.parametrize("T", [0, 4, 300])
def test_prompt_states_that_are_shifted(T):
    """h is h0 or apart from it; what is accepted is shown by the check after it (the workspace's, or the queries')."""
    d = _dims()
    size, h = d.B * d.H * d.dk * d.dv * 4, 0x10000000
    call = lambda h0, q: lq.load().lq_gdn_prefill_ragged(ct.byref(d), None, ct.c_void_p(h0), ct.c_void_p(h), T, q, A, A, A,
                                                         A, None, A, None, 0, None)
    for off in (16, size - 16, 16 - size, -16):
        assert call(h + off, A) == lq.LQ_ERR_OVERLAP
    if T:
        for off in (0, size, -size):
            assert call(h + off, None) == lq.LQ_ERR_NULL
