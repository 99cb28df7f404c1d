"""Host-only checks of the serving operators' entry points (prompts of the gated
delta rule, verification of drafted trees, rows of states moved): sizes, argument
errors with no HIP call, the binding's refusals, and the verification's rule itself."""
import ctypes as ct
import os
import random

import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.skipif(not os.path.exists(lq.LIB_PATH), reason="liblq.so not built")

A = ct.c_void_p(0x7000000)      # an aligned address that is never dereferenced
B4 = ct.c_void_p(0x7000004)
B2 = ct.c_void_p(0x7000002)
NAMES = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")


def _dims(**kw):
    base = dict(B=2, H=3, dk=128, dv=128, W=16, C=4, decay_mode=0, smooth=1, io_dtype=0)
    base.update(kw)
    return lq.lq_dims(*[base[n] for n in ("B", "H", "dk", "dv", "W", "C", "decay_mode", "smooth", "io_dtype")])


def _state(at=1, **kw):
    vals = {n: 0x10000000 * at + 0x1000000 * i for i, n in enumerate(NAMES)}
    vals.update(kw)
    return lq.lq_state(*[vals[n] for n in NAMES])


def test_prompt_argument_errors():
    L = lq.load()

    def call(d=None, st=None, h0=None, h=A, T=4, q=A, k=A, v=A, al=A, be=A, lens=None, o=A, ws=A, n=1 << 40):
        d = _dims() if d is None else d
        return L.lq_gdn_prefill_ragged(ct.byref(d), st, h0, h, T, q, k, v, al, be, lens, o, ws, n, None)

    assert L.lq_gdn_prefill_ragged(None, None, None, A, 4, A, A, A, A, A, None, A, None, 0, None) == lq.LQ_ERR_NULL
    assert call(_dims(B=0)) == lq.LQ_ERR_DIMS
    assert call(_dims(dk=96, dv=96)) == lq.LQ_ERR_UNSUPPORTED
    assert call(T=-1) == lq.LQ_ERR_POS
    assert call(T=(1 << 30) + 1) == lq.LQ_ERR_UNSUPPORTED
    assert call(_dims(B=1 << 12, H=(1 << 11) + 1, dk=16, dv=16)) == lq.LQ_ERR_UNSUPPORTED
    assert call(h=None) == lq.LQ_ERR_NULL and call(h=B4) == lq.LQ_ERR_ALIGN
    assert call(h0=B4) == lq.LQ_ERR_ALIGN and call(lens=B2) == lq.LQ_ERR_ALIGN
    for name in ("q", "k", "v", "al", "be"):
        assert call(**{name: None}) == lq.LQ_ERR_NULL
    for name in ("q", "k", "v", "o"):
        assert call(**{name: B4}) == lq.LQ_ERR_ALIGN
    assert call(al=B2) == lq.LQ_ERR_ALIGN and call(be=B2) == lq.LQ_ERR_ALIGN
    assert call(_dims(decay_mode=1), al=B4) == lq.LQ_ERR_ALIGN
    assert call(st=ct.byref(_state(sq=None))) == lq.LQ_ERR_NULL
    assert call(st=ct.byref(_state(comp_val=0x100004))) == lq.LQ_ERR_ALIGN


def test_prompt_workspace():
    L = lq.load()
    assert L.lq_gdn_workspace_bytes(None, 64) == 0
    assert lq.lq_gdn_workspace_bytes(_dims(dk=96, dv=96), 1 << 20) == 0
    for T in (-1, 0, 1, 4, (1 << 30) + 1):
        assert lq.lq_gdn_workspace_bytes(_dims(), T) == 0
    for kw in (dict(B=1, H=1), dict(), dict(B=1, H=16, io_dtype=1), dict(B=1, H=2, dk=64, dv=64),
               dict(B=1, H=2, dk=16, dv=16), dict(B=64, H=32), dict(B=1, H=16, decay_mode=1),
               dict(B=1, H=3, decay_mode=1, io_dtype=1, dk=64, dv=64)):
        d = _dims(**kw)
        sizes = [lq.lq_gdn_workspace_bytes(d, T) for T in
                 (1, 15, 64, 65, 100, 500, 511, 512, 513, 1000, 2000, 4095, 5000, 16384, 16385, 40000, 1 << 20)]
        assert sizes == sorted(sizes)
        need = lq.lq_gdn_workspace_bytes(d, 16384)
        if need:
            call = lambda ws, n: L.lq_gdn_prefill_ragged(ct.byref(d), None, None, A, 16384, A, A, A, A, A, None, A, ws,
                                                         n, None)
            assert call(None, need) == lq.LQ_ERR_NULL
            assert call(B4, need) == lq.LQ_ERR_ALIGN
            assert call(A, need - 1) == lq.LQ_ERR_WORKSPACE


def test_verify_argument_errors():
    L = lq.load()

    def call(d=None, pos=A, N=8, parent=A, token=A, V=100, t=A, t0=A, q=A, q0=A, rep=1, u=A, path=A, P=4, n_path=A,
             nxt=A, ws=A, n=1 << 40):
        d = _dims() if d is None else d
        return L.lq_tree_verify(ct.byref(d), pos, N, parent, token, V, t, t0, q, q0, rep, u, path, P, n_path, nxt, ws, n,
                                None)

    assert call(_dims(B=0)) == lq.LQ_ERR_DIMS
    for kw in (dict(N=0), dict(N=-1), dict(P=0), dict(P=9), dict(V=0), dict(V=-5), dict(rep=2), dict(rep=-1)):
        assert call(**kw) == lq.LQ_ERR_DIMS, kw
    for kw in (dict(N=65), dict(V=(1 << 30) + 1), dict(d=_dims(B=1 << 20), V=(1 << 16) + 1),
               dict(d=_dims(B=(1 << 21) + 1))):
        assert call(**kw) == lq.LQ_ERR_UNSUPPORTED, kw
    for name in ("pos", "parent", "token", "t", "u", "path", "n_path", "nxt"):
        assert call(**{name: None}) == lq.LQ_ERR_NULL, name
    for name in ("pos", "parent", "token", "t", "t0", "q", "q0", "u", "path", "n_path", "nxt"):
        assert call(**{name: B2}) == lq.LQ_ERR_ALIGN, name
    assert call(q0=None) == lq.LQ_ERR_NULL               # a draft with a target before the first node
    need = lq.lq_verify_workspace_bytes(_dims(), 8, 100)
    assert need > 0 and call(ws=None) == lq.LQ_ERR_NULL and call(ws=B4) == lq.LQ_ERR_ALIGN
    assert call(n=need - 1) == lq.LQ_ERR_WORKSPACE
    for a in ((None, 8, 100), (_dims(), 0, 100), (_dims(), 65, 100), (_dims(), 8, 0), (_dims(), 8, (1 << 30) + 1)):
        assert L.lq_verify_workspace_bytes(ct.byref(a[0]) if a[0] else None, a[1], a[2]) == 0


def test_gather_argument_errors():
    L = lq.load()

    def call(d=None, n=1, dst=None, src=None, rows=2, index=A, pos=A, pos_out=None):
        d = _dims() if d is None else d
        dst = [_state(1)] if dst is None else dst
        src = [_state(2)] if src is None else src
        pk = lambda x: (lq.lq_state * len(x))(*x) if x else None
        return L.lq_state_gather(ct.byref(d), n, pk(dst), pk(src), rows, index, pos, pos_out, None)

    assert call(_dims(H=0)) == lq.LQ_ERR_DIMS and call(n=0) == lq.LQ_ERR_DIMS and call(rows=0) == lq.LQ_ERR_DIMS
    assert call(_dims(H=(1 << 17) + 1, B=1)) == lq.LQ_ERR_UNSUPPORTED
    assert call(dst=[]) == lq.LQ_ERR_NULL and call(src=[]) == lq.LQ_ERR_NULL
    assert call(index=None) == lq.LQ_ERR_NULL and call(index=B2) == lq.LQ_ERR_ALIGN
    assert call(pos=B2) == lq.LQ_ERR_ALIGN and call(pos_out=B2) == lq.LQ_ERR_ALIGN
    for f in NAMES:
        assert call(dst=[_state(1, **{f: None})]) == lq.LQ_ERR_NULL, f
        at = 0x20000002 if f in ("comp_idx", "buf_g") else 0x20000004   # (those two are read in words of four bytes)
        assert call(src=[_state(2, **{f: at})]) == lq.LQ_ERR_ALIGN, f
    assert call(_dims(decay_mode=lq.LQ_DECAY_PER_KEY), src=[_state(2, buf_g=0x20000004)]) == lq.LQ_ERR_ALIGN
    # without positions only the codecs count
    assert call(dst=[_state(1, row_scale=None)], pos=None) == lq.LQ_ERR_NULL
    # overlaps: a shifted state, another number of rows in place, one array shared, two layers on one state
    assert call(src=[_state(1, sq=0x10000000 + 16)]) == lq.LQ_ERR_OVERLAP
    assert call(src=[_state(1)], rows=3) == lq.LQ_ERR_OVERLAP
    assert call(src=[_state(2, buf_m=0x10000000 + 0x6000000 + 16)]) == lq.LQ_ERR_OVERLAP
    assert call(src=[_state(1, buf_k=0x20000000)]) == lq.LQ_ERR_OVERLAP
    assert call(n=2, dst=[_state(1), _state(1)], src=[_state(2), _state(3)]) == lq.LQ_ERR_OVERLAP
    assert call(n=2, dst=[_state(1), _state(2)], src=[_state(2), _state(1)]) == lq.LQ_ERR_OVERLAP
    assert call(pos_out=A) == lq.LQ_ERR_OVERLAP          # index itself
    assert call(pos=ct.c_void_p(0x7100000), pos_out=ct.c_void_p(0x7100004)) == lq.LQ_ERR_OVERLAP
    assert call(index=ct.c_void_p(0x10000010)) == lq.LQ_ERR_OVERLAP
    for at in (0x10000010, 0x20000010):                  # positions written into a state
        assert call(pos_out=ct.c_void_p(at)) == lq.LQ_ERR_OVERLAP
    assert call(_dims(B=2049), src=[_state(1)], rows=2049) == lq.LQ_ERR_UNSUPPORTED
    assert b"overlap" in L.lq_status_str(lq.LQ_ERR_OVERLAP)


def test_binding_refuses():
    d = lq.make_dims(2, 3, 16, 16, 4, 1)
    st = lq.LayerState.allocate(d, "cpu")
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    i32 = lambda *s: z(*s, dt=torch.int32)
    with pytest.raises(ValueError):
        lq.lq_gdn_prefill_ragged(d, None, None, z(2, 3, 16, 16), 0, None, None, None, None, None)
    ok = dict(pos=i32(2), parent=i32(2, 4), token=i32(2, 4), target=z(4, 2, 9), u=z(5, 2), path=i32(2, 4),
              n_path=i32(2), next=i32(2))
    for name, x in (("parent", i32(2)), ("path", i32(2)), ("target", z(4, 2)), ("pos", None), ("token", None)):
        with pytest.raises(ValueError):
            lq.lq_tree_verify(d, **{**ok, name: x})
    with pytest.raises(ValueError):
        lq.lq_tree_verify(d, **ok)                       # host tensors
    with pytest.raises(ValueError):
        lq.lq_tree_verify(d, **ok, draft0=z(2, 9))
    with pytest.raises(ValueError):
        lq.lq_state_gather(st, st, i32(2))
    with pytest.raises(ValueError):
        lq.lq_state_gather([], [], i32(2))
    with pytest.raises(ValueError):
        lq.lq_state_gather([st], [st, st], i32(2))
    other = lq.LayerState.allocate(lq.make_dims(2, 3, 16, 16, 8, 1), "cpu")
    with pytest.raises(ValueError):
        lq.lq_state_gather(st, other, i32(2))


@pytest.mark.parametrize("replace", [True, False, None])
def test_the_rule_keeps_the_targets_distribution(replace):
    """The token after the last committed one (accepted or drawn) is distributed as the target has it,
    whatever the draft: frequencies of 40000 runs within 5 standard deviations."""
    rng = random.Random(11)
    V, n = 5, 40000
    p = torch.tensor([0.05, 0.4, 0.0, 0.3, 0.25], dtype=torch.float64)
    q = torch.tensor([0.3, 0.1, 0.2, 0.35, 0.05], dtype=torch.float64)
    target, draft = p.expand(3, V), q.expand(3, V)
    count = [0] * V
    for _ in range(n):
        left, tok = q.tolist(), []
        for _ in range(3):                               # three children of the root
            t = rng.choices(range(V), left)[0]
            tok.append(t)
            if replace is False:
                left[t] = 0.0
        if replace is None:
            tok = [rng.randrange(V) for _ in range(3)]   # looked up, chosen without the target
        u = [rng.random() for _ in range(4)]
        path, nxt, _ = R.verify([-1, -1, -1], tok, target, u, 1, target0=p,
                                draft=None if replace is None else draft, draft0=None if replace is None else q,
                                replace=replace is not False)
        count[tok[path[0]] if path else nxt] += 1
    for t in range(V):
        x = float(p[t])
        assert abs(count[t] / n - x) <= 5 * (x * (1 - x) / n) ** 0.5, (t, count)


def test_the_chunk_form_is_the_recurrence():
    """The chunk form (I + A) M = R of the prompt equals the token-by-token reference in 64 bits."""
    torch.manual_seed(4)
    T, B, H, d = 11, 1, 2, 8
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    for per_key in (False, True):
        q, k, v = unit(rnd(T, B, H, d)), unit(rnd(T, B, H, d)), rnd(T, B, H, d)
        alpha = torch.rand(*((T, B, H, d) if per_key else (T, B, H)), dtype=torch.float64) * 0.7 + 0.3
        beta = torch.rand(T, B, H, dtype=torch.float64)
        h0 = rnd(B, H, d, d)
        o, h = R.gdn_prefill(q, k, v, alpha, beta, h0)
        for hd in range(H):
            Q, K, V, be = q[:, 0, hd], k[:, 0, hd], v[:, 0, hd], beta[:, 0, hd]
            g = (alpha[:, 0, hd] if per_key else alpha[:, 0, hd, None].expand(T, d)).log().cumsum(0)
            E = (g[:, None] - g[None]).exp()
            rr = (K[:, None] * E * K[None]).sum(-1)
            aa = (Q[:, None] * E * K[None]).sum(-1)
            Am = be[:, None] * rr.tril(-1)
            M = torch.linalg.solve(torch.eye(T, dtype=torch.float64) + Am, be[:, None] * (V - (g.exp() * K) @ h0[0, hd]))
            assert torch.allclose((g.exp() * Q) @ h0[0, hd] + aa.tril() @ M, o[:, 0, hd], rtol=1e-10, atol=1e-10)
            H1 = g[-1].exp()[:, None] * h0[0, hd] + ((g[-1] - g).exp() * K).T @ M
            assert torch.allclose(H1, h[0, hd], rtol=1e-10, atol=1e-10)
