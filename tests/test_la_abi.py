"""Host-only checks of the linear-attention and tree entry points: sizes,
argument errors with no HIP call, the binding's refusals, and the 64-bit
references against the dense recurrence."""
import ctypes as ct
import os

import pytest

from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.skipif(not os.path.exists(lq.LIB_PATH), reason="liblq.so not built")

A = ct.c_void_p(0x7000000)      # an aligned address that is never dereferenced
B4 = ct.c_void_p(0x7000004)
B2 = ct.c_void_p(0x7000002)


def _dims(**kw):
    base = dict(B=2, H=3, dk=128, dv=128, W=16, C=4, decay_mode=0, smooth=1, io_dtype=0)
    base.update(kw)
    return lq.lq_dims(*[base[n] for n in ("B", "H", "dk", "dv", "W", "C", "decay_mode", "smooth", "io_dtype")])


def _state(**kw):
    names = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")
    vals = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    vals.update(kw)
    return lq.lq_state(*[vals[n] for n in names])


def test_prefill_argument_errors():
    L = lq.load()

    def call(d=None, st=None, h0=None, h=A, T=4, q=A, k=A, v=A, al=A, kind=0, lens=None, o=A, ws=None, n=0):
        d = _dims() if d is None else d
        return L.lq_la_prefill(ct.byref(d), st, h0, h, T, q, k, v, al, kind, lens, o, ws, n, None)

    assert L.lq_la_prefill(None, None, None, A, 4, A, A, A, A, 0, None, A, None, 0, None) == lq.LQ_ERR_NULL
    assert call(_dims(B=0)) == lq.LQ_ERR_DIMS
    assert call(_dims(decay_mode=1)) == lq.LQ_ERR_UNSUPPORTED
    assert call(_dims(dk=96, dv=96)) == lq.LQ_ERR_UNSUPPORTED
    assert call(kind=2) == lq.LQ_ERR_DIMS and call(kind=-1) == lq.LQ_ERR_DIMS
    assert call(T=-1) == lq.LQ_ERR_POS
    assert call(T=(1 << 30) + 1) == lq.LQ_ERR_UNSUPPORTED
    assert lq.lq_la_workspace_bytes(_dims(), (1 << 30) + 1) == 0
    assert call(h=None) == lq.LQ_ERR_NULL and call(h=B4) == lq.LQ_ERR_ALIGN
    assert call(h0=B4) == lq.LQ_ERR_ALIGN and call(lens=B2) == lq.LQ_ERR_ALIGN
    for name in ("q", "k", "v", "al"):
        assert call(**{name: None}) == lq.LQ_ERR_NULL
    for name in ("q", "k", "v", "o"):
        assert call(**{name: B4}) == lq.LQ_ERR_ALIGN
    assert call(al=B2) == lq.LQ_ERR_ALIGN
    assert call(st=ct.byref(_state(sq=None))) == lq.LQ_ERR_NULL
    assert call(st=ct.byref(_state(comp_val=0x100004))) == lq.LQ_ERR_ALIGN


def test_workspace_errors_and_sizes():
    L = lq.load()
    assert L.lq_la_workspace_bytes(None, 64) == 0
    assert lq.lq_la_workspace_bytes(_dims(decay_mode=1), 1 << 20) == 0
    for T in (-1, 0, 1):
        assert lq.lq_la_workspace_bytes(_dims(), T) == 0
    # never less for a longer prompt, and refused when short, missing or misaligned
    for kw in (dict(B=1, H=1), dict(), dict(B=1, H=16, io_dtype=1), dict(B=1, H=2, dk=64, dv=64),
               dict(B=1, H=2, dk=16, dv=16), dict(B=64, H=32)):
        d = _dims(**kw)
        sizes = [lq.lq_la_workspace_bytes(d, T) for T in
                 (1, 15, 64, 65, 100, 500, 511, 512, 513, 1000, 2000, 4095, 5000, 16384, 16385, 40000, 1 << 20)]
        assert sizes == sorted(sizes)
        T = 16384
        need = lq.lq_la_workspace_bytes(d, T)
        if need:
            call = lambda ws, n: L.lq_la_prefill(ct.byref(d), None, None, A, T, A, A, A, A, 0, None, A, ws, n, None)
            assert call(None, need) == lq.LQ_ERR_NULL
            assert call(B4, need) == lq.LQ_ERR_ALIGN
            assert call(A, need - 1) == lq.LQ_ERR_WORKSPACE
    assert b"workspace" in L.lq_status_str(lq.LQ_ERR_WORKSPACE)


def test_decode_argument_errors():
    L = lq.load()
    d, st = _dims(), _state()
    call = lambda dd, s, pos, *p: L.lq_la_decode_step(ct.byref(dd), s, pos, *p, None)
    ok = (A, A, A, A, 0, A)
    assert call(d, None, 0, *ok) == lq.LQ_ERR_NULL
    assert call(d, ct.byref(st), 16, *ok) == lq.LQ_ERR_WINDOW_FULL
    assert call(d, ct.byref(st), -1, *ok) == lq.LQ_ERR_POS
    assert call(_dims(decay_mode=1), ct.byref(st), 0, *ok) == lq.LQ_ERR_UNSUPPORTED
    assert call(d, ct.byref(st), 0, A, A, A, A, 2, A) == lq.LQ_ERR_DIMS
    assert call(d, ct.byref(st), 0, A, A, A, A, 1, None) == lq.LQ_ERR_NULL
    assert call(d, ct.byref(st), 0, A, B4, A, A, 0, A) == lq.LQ_ERR_ALIGN
    assert call(d, ct.byref(_state(buf_m=None)), 0, *ok) == lq.LQ_ERR_NULL
    rag = lambda dd, s, pos, *p: L.lq_la_decode_step_ragged(ct.byref(dd), s, pos, *p, None)
    assert rag(d, ct.byref(st), None, *ok) == lq.LQ_ERR_NULL
    assert rag(d, ct.byref(st), B2, *ok) == lq.LQ_ERR_ALIGN
    assert rag(_dims(decay_mode=1), ct.byref(st), A, *ok) == lq.LQ_ERR_UNSUPPORTED


def test_tree_argument_errors():
    L = lq.load()
    st = _state()

    def gdn(d=None, s=st, pos=A, N=8, parent=A, q=A, k=A, v=A, al=A, be=A, o=A, tm=A, tg=A):
        return L.lq_gdn_tree_step(ct.byref(_dims() if d is None else d), ct.byref(s), pos, N, parent, q, k, v, al, be,
                                  o, tm, tg, None)

    def la(d=None, s=st, pos=A, N=8, parent=A, q=A, k=A, v=A, al=A, kind=0, o=A, tm=A, tg=A):
        return L.lq_la_tree_step(ct.byref(_dims() if d is None else d), ct.byref(s), pos, N, parent, q, k, v, al, kind,
                                 o, tm, tg, None)

    for f in (gdn, la):
        assert f(N=0) == lq.LQ_ERR_DIMS and f(N=-3) == lq.LQ_ERR_DIMS
        assert f(N=65) == lq.LQ_ERR_UNSUPPORTED
        for name in ("pos", "parent", "q", "k", "v", "al", "o", "tm", "tg"):
            assert f(**{name: None}) == lq.LQ_ERR_NULL, name
        for name in ("pos", "parent", "al", "tg"):
            assert f(**{name: B2}) == lq.LQ_ERR_ALIGN, name
        for name in ("q", "k", "v", "o", "tm"):
            assert f(**{name: B4}) == lq.LQ_ERR_ALIGN, name
        assert f(s=_state(buf_g=None)) == lq.LQ_ERR_NULL
        assert f(d=_dims(dk=96, dv=96)) == lq.LQ_ERR_UNSUPPORTED
    assert gdn(be=None) == lq.LQ_ERR_NULL
    assert gdn(d=_dims(decay_mode=1), al=B4) == lq.LQ_ERR_ALIGN      # per-key rows: 16 bytes
    assert gdn(d=_dims(decay_mode=1), tg=B4) == lq.LQ_ERR_ALIGN
    assert la(d=_dims(decay_mode=1)) == lq.LQ_ERR_UNSUPPORTED
    assert la(kind=7) == lq.LQ_ERR_DIMS


def test_commit_argument_errors():
    L = lq.load()

    def call(d=None, s=None, pos=A, N=8, path=A, P=4, n_path=A, k=A, tm=A, tg=A):
        s = _state() if s is None else s
        return L.lq_tree_commit(ct.byref(_dims() if d is None else d), ct.byref(s), pos, N, path, P, n_path, k, tm,
                                tg, None)

    for kw in (dict(N=0), dict(P=0), dict(P=9), dict(N=-1, P=-1)):
        assert call(**kw) == lq.LQ_ERR_DIMS
    assert call(N=65) == lq.LQ_ERR_UNSUPPORTED
    for name in ("pos", "path", "n_path", "k", "tm", "tg"):
        assert call(**{name: None}) == lq.LQ_ERR_NULL, name
    for name in ("pos", "path", "n_path", "tg"):
        assert call(**{name: B2}) == lq.LQ_ERR_ALIGN, name
    for name in ("k", "tm"):
        assert call(**{name: B4}) == lq.LQ_ERR_ALIGN, name
    assert call(s=_state(buf_k=None)) == lq.LQ_ERR_NULL
    assert call(d=_dims(decay_mode=1), tg=B4) == lq.LQ_ERR_ALIGN


def test_binding_refuses_host_tensors():
    import torch
    d = lq.make_dims(2, 3, 16, 16, 4, 1)
    st = lq.LayerState.allocate(d, "cpu")
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    x, o = z(2, 3, 16), z(2, 3, 16)
    i32 = lambda *s: z(*s, dt=torch.int32)
    with pytest.raises(ValueError):
        lq.lq_la_decode_step(st, 0, x, x, x, z(3), o)
    with pytest.raises(ValueError):
        lq.lq_la_prefill(d, None, None, z(2, 3, 16, 16), 0, None, None, None, None)
    with pytest.raises(ValueError):
        lq.lq_gdn_tree_step(st, i32(2), i32(2), x, x, x, z(2, 3), z(2, 3), o, x, x)      # parent [B]
    with pytest.raises(ValueError):
        lq.lq_la_tree_step(st, i32(2), i32(2, 1), x[None], x[None], x[None], z(3), o[None], x, x)
    with pytest.raises(ValueError):
        lq.lq_tree_commit(st, i32(2), i32(2), i32(2), x[None], x, x)                     # path [B]


@pytest.mark.parametrize("rule", ["gdn", "kda", "la"])
def test_tree_reference_is_the_dense_recurrence(rule):
    """The context form of the references equals the delta rule (or plain linear
    attention) run on the dense 64-bit state along every node's path."""
    import torch
    import la_reference as R
    torch.manual_seed(3)
    B, H, d, W, N = 2, 2, 16, 4, 7
    gd = d if rule == "kda" else 1
    rnd = lambda *s: torch.randn(s, dtype=torch.float64)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    hb = rnd(B, H, d, d)
    bk, bm = unit(rnd(B, H, W, d)), rnd(B, H, W, d)
    bg = torch.rand(B, H, W, gd, dtype=torch.float64).neg().cumsum(2) * 0.2
    q, k, v = unit(rnd(N, B, H, d)), unit(rnd(N, B, H, d)), rnd(N, B, H, d)
    alpha = torch.rand(*((N, B, H, d) if rule == "kda" else (N, B, H)), dtype=torch.float64) * 0.5 + 0.5
    beta = None if rule == "la" else torch.rand(N, B, H, dtype=torch.float64)
    parent = [[-1, 0, 0, 2, -1, 3, 1], [-1, -5, 0, 1, 2, 4, 9]]
    pos = [3, 0]
    o, m, g, eo, em, here = R.tree(hb, bk, bm, bg, pos, parent, q, k, v, alpha, beta)
    assert here.tolist() == [[True] * 7, [True, False, True, False, True, True, False]]
    for b in range(B):
        h0 = hb[b].clone()
        if pos[b]:
            gl = bg[b, :, pos[b] - 1]
            h0 = gl.exp()[..., None] * h0
            for i in range(pos[b]):
                h0 = h0 + (bk[b, :, i] * (gl - bg[b, :, i]).exp())[..., None] * bm[b, :, i][:, None, :]
        hs = {-1: h0}
        for n in range(N):
            if not here[b, n]:
                continue
            al = alpha[n, b][..., None] if rule != "kda" else alpha[n, b]
            h = hs[parent[b][n]] * al[..., None]
            u = v[n, b]
            if beta is not None:
                u = beta[n, b][:, None] * (u - (h * k[n, b][..., None]).sum(1))
            hs[n] = h = h + k[n, b][..., None] * u[:, None, :]
            assert torch.allclose(m[b, :, n], u, rtol=1e-11, atol=1e-11)
            assert torch.allclose(o[n, b], (h * q[n, b][..., None]).sum(1), rtol=1e-11, atol=1e-11)
