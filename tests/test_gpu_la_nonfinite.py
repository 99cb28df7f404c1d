"""Infinities and NaN in drafted trees, their windows and states, and in the states before prompts: what is finite
by the definition is right, and what is not comes out as an infinity or NaN."""
import pytest
import torch

import la_reference as R
import test_gpu_la as G
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def near_where_finite(got, ref, bound, what, dtype=torch.float32):
    got, ref, bound = got.cpu(), ref.cpu(), bound.cpu()
    fine = torch.isfinite(ref)
    assert not bool(torch.isfinite(got[~fine]).any()), f"{what}: finite where the definition is not"
    G.near(got[fine], ref[fine], bound[fine], what, dtype)


KINDS = [(rule, io, d) for rule in ("gdn", "kda", "la") for io in ("f32", "bf16") for d in (16, 64, 128)]


@pytest.mark.parametrize("N", [16, 40])
@pytest.mark.parametrize("rule,io,d", KINDS)
def test_tree_tokens(rule, io, d, N):
    """Values, keys and queries of some nodes, in several rows; the tokens of absent nodes hold NaN."""
    B, H, W, per_key = 4, 2, 16, rule == "kda"
    pos = [3, 0, 16, 9]
    dims, st, hb, bk, bm, bg = G.make_state(d + N, B, H, d, W, 2, io, per_key, slots=pos)
    q, k, v, alpha, beta = G.tokens(d, (N, B, H), d, io, per_key)
    parent = [[G.SHAPES[s](n) for n in range(N)] for s in ("two chains", "mixed", "binary", "chain")]
    parent[0][7] = -2
    v[5, 0, 0, 3], v[N - 4, 1, 1, 2] = INF, -INF
    v[N - 1, 2, 0, 0] = NAN                              # a leaf
    k[6, 0, 1, 2], q[4, 1, 0, 1], q[N - 2, 2, 1, 5], k[N - 3, 3, 0, 9] = NAN, INF, NAN, INF
    ref = [x.clone() for x in (q, k, v, alpha, beta)]
    for x in (q, k, v, alpha, beta):
        x[7, 0] = NAN
    for x in ref[3:]:
        x[7, 0] = 1.0
    b = None if rule == "la" else beta
    o, tm, tg = G.run_tree(st, pos, parent, q, k, v, alpha, b)
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, *ref[:4], None if rule == "la" else ref[4])
    on = here.t()
    near_where_finite(o.cpu()[on], ro[on], eo[on], "o", q.dtype)
    on = here[:, None, :, None].expand_as(rm)
    near_where_finite(tm.cpu()[on], rm[on], em[on], "m")


@pytest.mark.parametrize("rule,io,d", KINDS)
def test_tree_window_and_state(rule, io, d):
    """A window's m reaches its column, a window's key every node, a column scale its column, of its row and head."""
    N, B, H, W, per_key = 20, 5, 2, 16, rule == "kda"
    pos = [4, 16, 7, 8, 5]
    dims, st, hb, bk, bm, bg = G.make_state(d, B, H, d, W, 2, io, per_key, slots=pos)
    q, k, v, alpha, beta = G.tokens(d + 5, (N, B, H), d, io, per_key)
    parent = [[G.SHAPES["mixed"](n) for n in range(N)] for _ in range(B)]
    bm[0, 0, 2, 3], bm[1, 1, 15, d - 1], bk[2, 0, 1, 4] = INF, NAN, NAN
    st.buf_m.copy_(bm), st.buf_k.copy_(bk)
    st.col_scale[3, 1, 6] = INF
    hb[3, 1, :, 6] = NAN
    b = None if rule == "la" else beta
    o, tm, tg = G.run_tree(st, pos, parent, q, k, v, alpha, b)
    ro, rm, rg, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, q, k, v, alpha, b)
    near_where_finite(o, ro, eo, "o", q.dtype)
    near_where_finite(tm, rm, em, "m")
    assert torch.isfinite(ro[:, 4]).all() and torch.isfinite(ro[:, 2, 1]).all() and not torch.isfinite(ro[:, 2, 0]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,T", [(16, 50), (64, 50), (128, 50), (16, 600), (64, 600), (128, 600), (128, 3)])
def test_prompt_start_state(d, T, io):
    """A value of the state before a prompt reaches its column of the outputs and itself."""
    c = G.prefill_case(d + T, 1, 3, d, T, io)
    q, k, v, alpha, h0 = c
    h0[0, 0, 2, 5], h0[0, 2, 7, 1] = INF, NAN
    o, h = G.run_prefill(*c, io)
    ro, rh, oa, ha = R.la_prefill(*c)
    b = R.c_of(d) + 2 * (T / 16 + 1) * R.U
    near_where_finite(h, rh, b * ha, "h")
    near_where_finite(o, ro, b * oa, "o", G.IO[io][1])
    assert int((~torch.isfinite(rh)).sum()) == 2 and not torch.isfinite(ro[:, 0, 0, 5]).any()
