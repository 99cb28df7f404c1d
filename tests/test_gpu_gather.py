"""Rows of states admitted, forked, permuted, compacted and cleared on the GPU: every
byte has to be the one that reading all rows before writing any gives."""
import random

import pytest
import torch

import serving_reference as R
from recurrent_state_quant_lq_amd import lq

pytestmark = pytest.mark.gpu
FIELDS = ("sq", "row_scale", "col_scale", "comp_idx", "comp_val", "buf_k", "buf_m", "buf_g")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lq.load()


def state(seed, B, H, d, W, C, per_key):
    dm = lq.make_dims(B, H, d, d, W, C, lq.LQ_DECAY_PER_KEY if per_key else lq.LQ_DECAY_SCALAR)
    st = lq.LayerState.allocate(dm)
    g = torch.Generator().manual_seed(seed)
    for f in FIELDS:
        t = getattr(st, f)
        if t.dtype == torch.float32:                       # any bits, NaN among them
            t.view(torch.int32).copy_(torch.randint(-2 ** 31, 2 ** 31 - 1, t.shape, generator=g))
        else:
            t.copy_(torch.randint(-127, 128, t.shape, generator=g))
    return st


def host(st):
    """Every array's bits."""
    return {f: (getattr(st, f).view(torch.int32) if getattr(st, f).dtype == torch.float32 else getattr(st, f)).cpu()
            for f in FIELDS}


def expect(dst, src, index, pos, C):
    want = R.gather(dst, src, index, pos, C)
    for b, i in enumerate(index):
        if i == -2:
            want["col_scale"][b] = 0x3f800000              # 1.0f
    return want


def same(st, want):
    got = host(st)
    for f in FIELDS:
        assert torch.equal(got[f], want[f]), f


MAPS = {
    "shift": lambda b, B, r: (b + 1) % B,                  # one cycle
    "back": lambda b, B, r: b - 1 if b else lq.LQ_ROW_CLEAR,
    "swap": lambda b, B, r: b ^ 1 if (b ^ 1) < B else b,
    "one": lambda b, B, r: B // 2,                         # every row the same
    "any": lambda b, B, r: r.randint(-2, B - 1),
    "none": lambda b, B, r: lq.LQ_ROW_KEEP,
    "clear": lambda b, B, r: lq.LQ_ROW_CLEAR if b % 2 else r.choice([-1, -3, B, B + 7, 2 ** 31 - 1, -2 ** 31]),
}


@pytest.mark.parametrize("kind", sorted(MAPS))
@pytest.mark.parametrize("B,H,d,W,C,per_key,windows", [
    (1, 1, 16, 1, 0, False, True), (5, 3, 128, 16, 4, False, True), (9, 1, 64, 13, 1, True, True),
    (33, 2, 16, 5, 8, False, True), (6, 2, 128, 32, 3, True, False), (300, 1, 16, 4, 2, False, True),
    (2048, 1, 16, 2, 1, False, True), (70, 9, 64, 16, 4, False, True)])
def test_in_place(B, H, d, W, C, per_key, windows, kind):
    st = state(B + d, B, H, d, W, C, per_key)
    before = host(st)
    rng = random.Random(B)
    index = [MAPS[kind](b, B, rng) for b in range(B)]
    pos = [rng.choice([0, 1, W // 2, W, W + 5, -3]) for _ in range(B)] if windows else None
    p = None if pos is None else torch.tensor(pos, dtype=torch.int32).cuda()
    po = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    lq.lq_state_gather(st, st, torch.tensor(index, dtype=torch.int32).cuda(), p, po)
    same(st, expect(before, before, index, pos, C))
    assert po.tolist() == [0 if i == -2 else (pos[i] if pos else 0) if 0 <= i < B else 99 for i in index]


@pytest.mark.parametrize("B,S,H,d,W,C,per_key", [(4, 9, 3, 128, 16, 4, False), (70, 2, 1, 16, 7, 5, True),
                                                 (1, 1, 2, 64, 32, 0, False), (5000, 3, 1, 16, 1, 1, False)])
def test_from_another_batch(B, S, H, d, W, C, per_key):
    dst, src = state(1, B, H, d, W, C, per_key), state(2, S, H, d, W, C, per_key)
    a, b = host(dst), host(src)
    rng = random.Random(3)
    index = [rng.randint(-3, S) for _ in range(B)]
    pos = [rng.randint(0, W) for _ in range(S)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    lq.lq_state_gather(dst, src, i32(index), i32(pos))
    same(dst, expect(a, b, index, pos, C))
    same(src, b)


@pytest.mark.parametrize("layers", [1, 2, 24, 25, 49])
def test_layers_at_once(layers):
    B, H, d, W, C = 6, 2, 16, 4, 2
    dst = [state(l, B, H, d, W, C, False) for l in range(layers)]
    src = [state(100 + l, B, H, d, W, C, False) if l % 2 == 0 else dst[l] for l in range(layers)]   # some in place
    a, b = [host(x) for x in dst], [host(x) for x in src]
    index, pos = [3, 0, -2, 5, -1, 1], [0, 4, 1, 2, 3, 0]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    po = i32([9] * B)
    lq.lq_state_gather(dst, src, i32(index), i32(pos), po)
    for l in range(layers):
        same(dst[l], expect(a[l], b[l], index, pos, C))
    assert po.tolist() == [2, 0, 0, 0, 9, 4]


@pytest.mark.parametrize("per_key", [False, True])
def test_layers_of_one_allocation(per_key):
    """Arrays of all layers in one tensor: a layer's compensator indices and log decays start at any word."""
    layers, B, S, H, d, W, C = 3, 5, 3, 1, 16, 3, 1
    parts = [[state(9 * i + l, n, H, d, W, C, per_key) for l in range(layers)] for i, n in ((0, B), (1, S))]
    sts = []
    for states in parts:
        whole = {f: torch.stack([getattr(x, f) for x in states]) for f in FIELDS}
        sts.append([lq.LayerState(x.dims, *[whole[f][l] for f in FIELDS]) for l, x in enumerate(states)])
    assert any(x.comp_idx.data_ptr() % 16 for x in sts[0]) and (per_key or any(x.buf_g.data_ptr() % 16 for x in sts[0]))
    index, pos = [2, lq.LQ_ROW_CLEAR, 0, lq.LQ_ROW_KEEP, 2], [3, 1, 2]
    dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    want = [expect(host(x), host(y), index, pos, C) for x, y in zip(*sts)]
    lq.lq_state_gather(*sts, dev(index), dev(pos))
    for x, w in zip(sts[0], want):
        same(x, w)


def test_rows_of_views():
    """Two halves of one batch as states of their own."""
    st = state(5, 8, 3, 64, 8, 4, False)
    a = host(st)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    lq.lq_state_gather(st.rows(0, 4), st.rows(4, 8), i32([3, -1, 0, -2]), i32([8, 1, 0, 3]))
    half = lambda x, lo, hi: {f: t[lo:hi] for f, t in x.items()}
    same(st.rows(0, 4), expect(half(a, 0, 4), half(a, 4, 8), [3, -1, 0, -2], [8, 1, 0, 3], 4))
    same(st.rows(4, 8), half(a, 4, 8))
    with pytest.raises(lq.LQError):                        # halves that share rows
        lq.lq_state_gather(st.rows(0, 4), st.rows(2, 6), i32([0, 1, 2, 3]))


def test_cleared_rows_are_the_codec_of_a_zero_state():
    for C in (0, 3):
        st = state(6, 4, 2, 64, 8, C, False)
        want = lq.LayerState.allocate(st.dims)
        lq.lq_gdn_state_quantize(want, torch.zeros(4, 2, 64, 64, device="cuda"))
        lq.lq_state_gather(st, st, torch.full((4,), lq.LQ_ROW_CLEAR, dtype=torch.int32, device="cuda"))
        for f in FIELDS[:5]:
            if C or not f.startswith("comp"):
                assert torch.equal(getattr(st, f).view(torch.uint8), getattr(want, f).view(torch.uint8)), f


def test_graphs_and_streams():
    """A captured in-place gather with other maps every replay, and two gathers of disjoint states at once."""
    B, H, d, W, C = 12, 4, 128, 16, 4
    st = state(7, B, H, d, W, C, False)
    index = torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    index.fill_(-1)
    g = torch.cuda.CUDAGraph()
    lq.lq_state_gather(st, st, index, pos)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lq.lq_state_gather(st, st, index, pos)
    rng = random.Random(4)
    for _ in range(4):
        a = host(st)
        idx, p = [rng.randint(-2, B - 1) for _ in range(B)], [rng.randint(0, W) for _ in range(B)]
        index.copy_(torch.tensor(idx, dtype=torch.int32))
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same(st, expect(a, a, idx, p, C))
    a = host(st)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    one, two, pz = i32([1, 0, 3, 2, 5, 4]), i32([5, 4, 3, 2, 1, 0]), i32([16] * 6)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    h1, h2 = st.rows(0, 6), st.rows(6, 12)
    lq.lq_state_gather(h1, h1, one, pz, stream=s1)
    lq.lq_state_gather(h2, h2, two, pz, stream=s2)
    torch.cuda.synchronize()
    half = lambda x, lo, hi: {f: t[lo:hi] for f, t in x.items()}
    same(h1, expect(half(a, 0, 6), half(a, 0, 6), one.tolist(), [16] * 6, C))
    same(h2, expect(half(a, 6, 12), half(a, 6, 12), two.tolist(), [16] * 6, C))


def test_refusals():
    st = state(8, 4, 2, 16, 4, 1, False)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    idx = i32([0, 1, 2, 3])
    for args in ((idx.long(),), (idx[:3],), (idx, idx.long()), (idx, idx[:2]), (idx, None, idx[:2]), (idx.cpu(),)):
        with pytest.raises(ValueError):
            lq.lq_state_gather(st, st, *args)
    with pytest.raises(lq.LQError):
        lq.lq_state_gather(st, st, idx, idx, idx)          # pos_out is an input
    other = state(9, 4, 2, 16, 4, 2, False)
    with pytest.raises(ValueError):
        lq.lq_state_gather(st, other, idx)
