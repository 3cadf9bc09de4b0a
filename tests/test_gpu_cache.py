"""GPU parity of decoding over a paged cache: block planning (whole numbers, equal),
attention of one token, chains and trees of drafts (against the fp64 oracle), and
whole decoding runs against dense attention.

Tolerance of o, elementwise: the weights are rounded to bf16 for the product
with V (2^-8 of each, so 2^-8 of the weighted mean of |v|, which the oracle
gives) and their fp32 errors are far smaller -- a score is a sum of D <= 128
products in fp32, off by at most 2^-20 (about D 2^-24 / 8) of the sum of |q k|
/ sqrt(D) < 64 in these inputs, so a weight by 2^-14, the exponential's and the
joins' errors below that: 2^-12 of the same mean in all; the result is rounded
to bf16 (2^-8 of it).  lse: the scores' 2^-14 and 2^-20 of its size.
"""
import numpy as np
import pytest
import torch

import oracle.cache_ref as cr
from sparse_attention_attn_b200 import inputs as I
from tests.parity_util import to64

pytestmark = pytest.mark.gpu


def s2():
    import sparse_attention_attn_b200
    return sparse_attention_attn_b200


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ planning

def _plan_case(R, ctx_hi, new_hi, bs, tree, seed, pad=0, short=0, width=None):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, ctx_hi + 1, R), rng.integers(0, new_hi + 1, R)
    have, need = -(-ctx // bs), -(-(ctx + new) // bs)
    width = int(need.max()) + 1 if width is None else width
    ids = rng.permutation(int(need.sum()) + 5)
    tab, at = np.full((R, width), -1), 0
    for r in range(R):
        n = min(have[r], width)
        tab[r, :n] = ids[at:at + n]
        at += n
    free = ids[at:]
    free = free[:max(0, int((need - have).sum()) - short)] if short else free
    T = max(1, int(new.sum()) + pad)
    parents = None
    if tree:
        parents = np.full(T, -1)
        t = 0
        for n in new:
            for j in range(n):
                parents[t] = max(-1, j - rng.integers(1, 7))
                t += 1
    return ctx, new, tab, free, T, parents


def _check_plan(ctx, new, tab, free, bs, T, parents):
    d_tab = i32(tab)
    p = s2().cache_plan(i32(ctx), i32(new), d_tab, i32(free), bs, T, None if parents is None else i32(parents))
    torch.cuda.synchronize()
    cu, pos, slots, mask, counts, out = cr.plan(ctx, new, tab, free, bs, T, parents)
    for name, got, want in (("cu", p.cu_seqlens, cu), ("pos", p.positions, pos), ("slots", p.slots, slots),
                            ("counts", p.counts, counts), ("tables", d_tab, out)):
        assert np.array_equal(got.cpu().numpy(), want), name
    assert (p.mask is None) == (parents is None)
    if parents is not None:
        assert np.array_equal(p.mask.cpu().numpy(), mask)


@pytest.mark.parametrize("R,ctx_hi,new_hi,bs,tree,pad", [
    (1, 0, 1, 16, False, 0), (1, 100, 1, 16, False, 3), (3, 40, 64, 16, True, 0), (64, 8000, 1, 16, False, 0),
    (300, 500, 64, 32, True, 300), (1500, 30, 3, 128, False, 17), (5, 3000, 3000, 256, False, 0), (7, 20, 90, 1, True, 5),
    (2100, 50, 40, 24, True, 1), (4, 0, 0, 16, False, 2),
])
def test_plan_against_oracle(R, ctx_hi, new_hi, bs, tree, pad):
    ctx, new, tab, free, T, parents = _plan_case(R, ctx_hi, new_hi, bs, tree, R + bs, pad)
    _check_plan(ctx, new, tab, free, bs, T, parents)


def test_plan_when_blocks_run_out():
    ctx, new, tab, free, T, parents = _plan_case(40, 200, 50, 16, False, 3, short=7)
    _check_plan(ctx, new, tab, free, 16, T, parents)          # the free list
    ctx, new, tab, free, T, parents = _plan_case(40, 200, 50, 16, True, 4, width=9)
    _check_plan(ctx, new, tab, free, 16, T, parents)          # the table's width
    _check_plan(ctx, new, tab, free[:0], 16, T, parents)      # no free block at all
    _check_plan(ctx, new, tab, free, 16, max(1, T - 100), None)  # fewer places than tokens


def test_plan_odd_lengths_and_parents():
    ctx, new, tab, free, T, parents = _plan_case(6, 30, 70, 16, True, 5)
    ctx[2], new[3] = -5, -7   # count as 0
    parents = np.full(400, -1)
    parents[::3], parents[1::5] = 40, -9   # later than the draft, or negative: hangs on the context
    parents[2::4] = 0
    _check_plan(ctx, new, tab, np.arange(500, 600), 16, 400, parents)


# ------------------------------------------------------------------ attention

@pytest.fixture(params=["cluster", "dec", "tc"])
def kernel(request):
    """Both attention kernels, whichever the call's sizes would pick."""
    from sparse_attention_attn_b200 import _lib
    _lib.s2attn_set_tile_override("cache=" + request.param)
    yield request.param
    _lib.s2attn_set_tile_override(None)


def _batch(lens, H, Hkv, D, bs, masks, seed, pad=0, spare=2, poison=True):
    """lens: (ctx, new) a request.  Unused rows of the cache hold NaN."""
    rng = np.random.default_rng(seed)
    R, need = len(lens), [-(-(c + n) // bs) for c, n in lens]
    nb = sum(need) + spare
    ids = rng.permutation(nb)
    width = max(1, max(need)) + 1
    tab, at = np.full((R, width), -7), 0
    kc = torch.full((nb, bs, Hkv, D), float("nan") if poison else 0.0, dtype=torch.bfloat16)
    vc = kc.clone()
    reqs, T = [], sum(n for _, n in lens) + pad
    q = I.randn_bf16((max(T, 1), H, D), seed)
    for r, (c, n) in enumerate(lens):
        tab[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        k, v = I.randn_bf16((c + n, Hkv, D), seed + 10 + r), I.randn_bf16((c + n, Hkv, D), seed + 500 + r)
        p = np.arange(c + n)
        kc[tab[r, p // bs], p % bs], vc[tab[r, p // bs], p % bs] = k, v
        reqs.append((k, v))
    cu = np.concatenate(([0], np.cumsum([n for _, n in lens])))
    return dict(q=q, kc=kc, vc=vc, tab=tab, cu=cu, lens=lens, reqs=reqs, masks=masks, T=max(T, 1))


def _call(b, **kw):
    mask = None
    if b["masks"] is not None:
        m = np.zeros(b["T"], np.uint64)
        for r, x in enumerate(b["masks"]):
            m[b["cu"][r]:b["cu"][r + 1]] = x
        mask = torch.from_numpy(m.view(np.int64)).cuda()
    return s2().cache_attention(b["q"].cuda(), b["kc"].cuda(), b["vc"].cuda(), i32(b["tab"]),
                                i32([c for c, _ in b["lens"]]), i32(b["cu"]), mask=mask, **kw)


def _check(b, o, lse, rows=None):
    o, lse, t_end = to64(o), to64(lse), b["cu"][-1]
    for r, (c, n) in enumerate(b["lens"]):
        if n == 0:
            continue
        t0 = b["cu"][r]
        k, v = (to64(x) for x in b["reqs"][r])
        see = cr.visible(n, None if b["masks"] is None else b["masks"][r])
        want, want_l, mag = cr.attention(to64(b["q"])[t0:t0 + n], k, v, c, see)
        got, got_l = o[t0:t0 + n], lse[:, t0:t0 + n]
        bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * mag
        assert not bad.any(), (r, c, n, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
        empty = np.isneginf(want_l)
        assert np.array_equal(np.isneginf(got_l), empty)
        assert np.all(np.abs(got_l[~empty] - want_l[~empty]) <= 2.0 ** -14 + 2.0 ** -20 * np.abs(want_l[~empty]))
    return t_end


def _tree_masks(lens, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    out = []
    for _, n in lens:
        m = np.zeros(n, np.uint64)
        for j in range(min(n, 64)):
            up = j - rng.integers(1, 6)
            m[j] = np.uint64(1 << j) | (m[up] if up >= 0 else np.uint64(0))
        m[rng.random(n) < drop] = np.uint64(0)
        out.append(m)
    return out


LENS = {
    "one": [(0, 1)], "first-key": [(1, 1)], "tile-edges": [(63, 1), (64, 1), (65, 1), (127, 1), (128, 1), (15, 1), (16, 1)],
    "long": [(5000, 1)], "ragged": [(17, 3), (700, 1), (0, 5), (333, 2), (1, 1), (64, 64)], "gaps": [(10, 0), (30, 2), (0, 0), (5, 4), (9, 0)],
    "chunk": [(100, 200), (0, 130)], "many": [(3 * i % 97, i % 3) for i in range(300)], "sparse": [(40 + i, int(i % 71 == 5)) for i in range(500)], "drafts": [(900, 61), (127, 64), (3, 7)],
}


@pytest.mark.parametrize("H,Hkv,D,bs", [(4, 4, 64, 16), (8, 2, 128, 32), (6, 2, 64, 64), (16, 1, 128, 256)])
@pytest.mark.parametrize("lens", list(LENS), ids=list(LENS))
def test_chain_attention_against_oracle(kernel, lens, H, Hkv, D, bs):
    b = _batch(LENS[lens], H, Hkv, D, bs, None, 7, pad=3)
    out = torch.full((b["T"], H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, b["T"]), 9.0, device="cuda")
    o, l = _call(b, out=out, lse=lse)
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    t = _check(b, o, l)
    assert (o[t:] == 5.0).all() and (l[:, t:] == 9.0).all()  # rows of no request as they were


@pytest.mark.parametrize("pages", [0, 600, 1100])  # wide tables: the host knows no lengths, only their limit
@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 64), (9, 9, 128), (24, 24, 128), (33, 33, 64), (16, 1, 128), (24, 8, 128)])
@pytest.mark.parametrize("ctx,new,tree", [(0, 0, False), (0, 1, False), (63, 1, False), (64, 1, True), (1023, 2, False), (1030, 2, True), (2600, 1, False)])
def test_single_request(ctx, new, tree, H, Hkv, D, pages):
    """Whichever form the sizes pick, twice the same bits, rows behind left as they were."""
    b = _batch([(ctx, new)], H, Hkv, D, 16, _tree_masks([(ctx, new)], 4) if tree else None, 23, pad=0 if new else 2)
    b["tab"] = np.pad(b["tab"], ((0, 0), (0, max(0, pages - b["tab"].shape[1]))), constant_values=-1)
    outs = []
    for _ in range(2):
        out = torch.full((b["T"], H, D), 5.0, dtype=torch.bfloat16, device="cuda")
        outs.append(_call(b, out=out, lse=torch.full((H, b["T"]), 9.0, device="cuda")))
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    t = _check(b, *outs[0])
    assert (outs[0][0][t:] == 5.0).all() and (outs[0][1][:, t:] == 9.0).all()


@pytest.mark.parametrize("pages", [0, 70, 300])  # up to 1024 keys a CTA in clusters, else equal runs
@pytest.mark.parametrize("R,H,Hkv,D", [(2, 8, 4, 128), (5, 12, 6, 64), (9, 28, 7, 128), (16, 8, 8, 64), (37, 8, 8, 128), (75, 8, 8, 64), (129, 4, 2, 64)])
def test_batches_of_few_items(R, H, Hkv, D, pages):
    """Every size of cluster, ragged lengths with requests that have no new token or several."""
    lens = [((37 * i) % 900, (1, 1, 0, 2, 1)[i % 5]) for i in range(R)]
    b = _batch(lens, H, Hkv, D, 16, _tree_masks(lens, 6) if pages == 70 else None, 29, pad=2)
    b["tab"] = np.pad(b["tab"], ((0, 0), (0, max(0, pages - b["tab"].shape[1]))), constant_values=-1)
    out = torch.full((b["T"], H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    o, l = _call(b, out=out, lse=torch.full((H, b["T"]), 9.0, device="cuda"))
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    t = _check(b, o, l)
    assert (o[t:] == 5.0).all() and (l[:, t:] == 9.0).all()


@pytest.mark.parametrize("H,Hkv,D,bs", [(40, 1, 64, 16), (128, 1, 128, 64)])
@pytest.mark.parametrize("lens", ["one", "tile-edges", "ragged", "gaps"])
def test_more_than_16_heads_a_kv_head(lens, H, Hkv, D, bs):
    b = _batch(LENS[lens], H, Hkv, D, bs, None, 8)
    _check(b, *_call(b))


@pytest.mark.parametrize("H,Hkv,D,bs", [(4, 4, 128, 16), (32, 4, 64, 128), (5, 1, 128, 64)])
@pytest.mark.parametrize("lens,drop", [("drafts", 0.0), ("ragged", 0.0), ("drafts", 0.4), ("one", 1.0), ("tile-edges", 1.0)])
def test_tree_attention_against_oracle(kernel, lens, drop, H, Hkv, D, bs):
    b = _batch(LENS[lens], H, Hkv, D, bs, _tree_masks(LENS[lens], 3, drop), 11)
    o, l = _call(b)
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    _check(b, o, l)


def test_row_without_any_key_is_zero(kernel):
    b = _batch([(0, 3), (0, 1)], 4, 2, 128, 16, [np.array([0, 2, 0], np.uint64), np.array([0], np.uint64)], 13)
    o, l = _call(b)
    assert (o[[0, 2, 3]] == 0).all() and torch.isneginf(l[:, [0, 2, 3]]).all()
    _check(b, o, l)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (8, 2, 128), (16, 1, 128)])
def test_non_finite_drafts_reach_only_the_rows_that_see_them(kernel, H, Hkv, D, tree):
    lens = [(37, 6), (126, 5), (0, 2), (255, 1), (70, 40)]
    masks = _tree_masks(lens, 5) if tree else None
    if tree:
        masks[2] = np.array([2, 1], np.uint64)   # each sees the other one only
        masks[3] = np.array([0], np.uint64)      # sees the context only
    b = _batch(lens, H, Hkv, D, 16, masks, 19)
    for r, (c, n) in enumerate(lens):
        k, v = b["reqs"][r]
        for j, col, x in ((n - 1, 3, float("nan")), (n // 2, 10, float("inf")), (n // 2, D - 1, -float("inf"))):
            v[c + j, -1, col] = x
        if n > 5:
            k[c + 4, 0, 7] = float("nan")        # the scores of those that see it
        p = np.arange(c + n)
        b["kc"][b["tab"][r, p // 16], p % 16], b["vc"][b["tab"][r, p // 16], p % 16] = k, v
    o, l = (to64(x) for x in _call(b))
    for r, (c, n) in enumerate(lens):
        t0 = b["cu"][r]
        with np.errstate(invalid="ignore"):
            want, want_l, mag = cr.attention(to64(b["q"])[t0:t0 + n], *(to64(x) for x in b["reqs"][r]), c,
                                             cr.visible(n, None if masks is None else masks[r]))
        got = o[t0:t0 + n]
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        fine = np.isfinite(want)
        g, w = got[fine], want[fine]
        assert np.all(np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -12) * mag[fine])
        assert np.array_equal(np.isnan(l[:, t0:t0 + n]), np.isnan(want_l))


def test_bits_of_drafts_that_do_not_exist_are_ignored(kernel):
    b = _batch([(40, 5)], 4, 2, 64, 16, [np.full(5, 0xFFFFFFFFFFFFFFFF, np.uint64)], 14)
    o, l = _call(b)
    _check(b, o, l)


def test_same_bits_every_time_and_on_another_stream(kernel):
    b = _batch([(4000, 2), (77, 1), (0, 9)], 16, 4, 128, 64, None, 15)
    o, l = _call(b)
    torch.cuda.synchronize()
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(255)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        o2, l2 = _call(b, workspace=ws)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_blocks_out_of_range_are_reported_and_read_as_zeros(kernel):
    b = _batch([(40, 1), (20, 1)], 4, 2, 64, 16, None, 16)
    good, _ = _call(b)
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    b["tab"][0, 1] = 10 ** 6
    o, l = _call(b)
    assert s2().device_status() == 7 and s2().device_status() == 0
    assert torch.equal(o[1], good[1])
    k, v = (x.clone() for x in b["reqs"][0])
    k[16:32] = 0
    v[16:32] = 0
    b["reqs"][0] = (k, v)
    _check(b, o, l)


def test_offsets_beyond_32_bits(kernel):
    """A cache of more than 2^31 elements, the blocks at its far end."""
    Hkv, D, bs, nb = 8, 128, 256, 9000   # 2.36e9 elements each
    b = _batch([(600, 2), (256, 1)], 16, Hkv, D, bs, None, 17, spare=0)
    small = b["kc"].shape[0]
    kc = torch.empty(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    kc[nb - small:], vc[nb - small:] = b["kc"].cuda(), b["vc"].cuda()
    tab = np.where(b["tab"] >= 0, b["tab"] + nb - small, b["tab"])
    o, l = s2().cache_attention(b["q"].cuda(), kc, vc, i32(tab), i32([600, 256]), i32(b["cu"]))
    _check(b, o, l)
    new = I.randn_bf16((2, Hkv, D), 3).cuda()
    slots = [nb * bs - 1, nb * bs - 700]
    s2().cache_append(I.randn_bf16((2, 16, D), 4).cuda(), new, new, s2().rope_table(4, D, 1.0), i32([0, 0]), i32(slots),
                      kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(vc.view(-1, Hkv, D)[slots], new) and torch.equal(kc.view(-1, Hkv, D)[slots], new)
    assert s2().device_status() == 0


# ------------------------------------------------------------------ whole runs

def _decode(chunks, x, weights, table, bs, H, Hkv, D, nb=64, width=40):
    """Feeds x = (q, k, v) [N, heads, D] of two requests (the second in other
    chunk sizes) through plan, append and attention; returns o of each."""
    kc = torch.full((nb, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    tab = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(nb, device="cuda").int()
    ctx, outs, at = [0, 0], [[], []], [0, 0]
    for new in chunks:
        T = sum(new) + 2
        p = s2().cache_plan(i32(ctx), i32(new), tab, free, bs, T)
        rows = [x[r][i][at[r]:at[r] + new[r]] for i in range(3) for r in range(2)]
        q, k, v = (torch.cat((rows[2 * i], rows[2 * i + 1], torch.zeros_like(x[0][i][:2]))) for i in range(3))
        q = s2().cache_append(q, k, v, table, p.positions, p.slots, kc, vc, *weights)
        o, _ = s2().cache_attention(q, kc, vc, tab, i32(ctx), p.cu_seqlens)
        taken, needed, total, lost = p.counts.tolist()
        assert taken == needed and total == sum(new) and lost == 0
        free = free[taken:]
        outs[0].append(o[:new[0]])
        outs[1].append(o[new[0]:new[0] + new[1]])
        for r in range(2):
            ctx[r] += new[r]
            at[r] += new[r]
    return [torch.cat(o) for o in outs]


@pytest.mark.parametrize("norm", [True, False])
def test_decoding_in_steps_is_dense_attention(norm):
    N, H, Hkv, D, bs = 256, 8, 2, 128, 16
    x = [[I.randn_bf16((N, h, D), 100 * r + i).cuda() for i, h in enumerate((H, Hkv, Hkv))] for r in range(2)]
    table = s2().rope_table(N, D, 0.5)
    w = [(1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(i))).cuda() for i in (1, 2)] if norm else [None, None]
    chunks = [(100, 1), (1, 1), (1, 70), (1, 0), (0, 3), (64, 101), (89, 80)]
    outs = _decode(chunks, x, w, table, bs, H, Hkv, D)
    for r in range(2):
        q, k, v = (t[None] for t in x[r])
        if norm:
            o = s2().dense_causal_attn(*s2().qknorm_rope_forward(q, k, *w, table), v)
        else:
            o = s2().dense_causal_attn(s2().rope_apply(q, table), s2().rope_apply(k, table), v)
        # both round the weights (2^-8 of the mean of |v|) and the result: twice the one-sided tolerance
        a, b = to64(outs[r]), to64(o[0])
        assert np.all(np.abs(a - b) <= 2 * 2.0 ** -8 * np.abs(b) + 2 * (2.0 ** -8 + 2.0 ** -12) * np.abs(to64(v)).max())
        assert np.linalg.norm(a - b) <= 5e-3 * np.linalg.norm(b)


def test_drafted_tree_matches_its_paths():
    """A tree of drafts in one call gives every draft what decoding its path alone gives."""
    H, Hkv, D, bs, ctx = 8, 4, 64, 16, 37
    parents = [-1, -1, 0, 0, 1, 2, 2, 4]
    n = len(parents)
    kc = I.randn_bf16((12, bs, Hkv, D), 1).cuda()
    vc = I.randn_bf16((12, bs, Hkv, D), 2).cuda()
    table = s2().rope_table(64, D, 1.0)
    q, k, v = (I.randn_bf16((n, h, D), 5 + h) .cuda() for h in (H, Hkv, Hkv))
    tab0 = torch.tensor([[3, 9, 0, -1, -1]], dtype=torch.int32, device="cuda")
    free = i32([1, 2, 4, 5])

    def step(idx, par):
        tab, k2, v2 = tab0.clone(), kc.clone(), vc.clone()
        p = s2().cache_plan(i32([ctx]), i32([len(idx)]), tab, free, bs, len(idx), None if par is None else i32(par))
        qq = s2().cache_append(q[idx], k[idx], v[idx], table, p.positions, p.slots, k2, v2)
        return s2().cache_attention(qq, k2, v2, tab, i32([ctx]), p.cu_seqlens, mask=p.mask)

    o, lse = step(list(range(n)), parents)
    for j in range(n):
        path = [j]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        po, pl = step(path, None)
        d = (to64(o[j]) - to64(po[-1]))
        assert np.abs(d).max() <= 2 * (2.0 ** -8 * np.abs(to64(po[-1])).max() + 2.0 ** -8 * 4.0)
        assert np.abs(to64(lse[:, j]) - to64(pl[:, -1])).max() <= 2.0 ** -13


def test_captured_step_follows_new_lengths(kernel):
    """One captured step (plan, append, attention) replayed for growing contexts."""
    H, Hkv, D, bs, R = 8, 2, 128, 16, 3
    kc = I.randn_bf16((64, bs, Hkv, D), 1).cuda()
    vc = I.randn_bf16((64, bs, Hkv, D), 2).cuda()
    table = s2().rope_table(512, D, 1.0)
    tab = torch.arange(60, dtype=torch.int32, device="cuda").view(R, 20).contiguous()
    free = i32([60, 61, 62, 63])
    ctx, new = i32([5, 100, 250]), i32([1, 1, 1])
    q, k, v = (I.randn_bf16((4, h, D), 5 + h).cuda() for h in (H, Hkv, Hkv))

    def step(kc, vc):
        p = s2().cache_plan(ctx, new, tab, free, bs, 4)
        qq = s2().cache_append(q, k, v, table, p.positions, p.slots, kc, vc)
        o = torch.zeros_like(q)
        return s2().cache_attention(qq, kc, vc, tab, ctx, p.cu_seqlens, out=o, lse=torch.zeros(H, 4, device="cuda"))

    step(kc.clone(), vc.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    kg, vg = kc.clone(), vc.clone()
    with torch.cuda.graph(g):
        cap = step(kg, vg)
    ke, ve = kc.clone(), vc.clone()
    for lens in ([5, 100, 250], [6, 101, 251], [300, 0, 17], [1, 318, 64]):
        ctx.copy_(i32(lens))
        g.replay()
        want = step(ke, ve)
        torch.cuda.synchronize()
        assert torch.equal(cap[0], want[0]) and torch.equal(cap[1], want[1]) and torch.equal(kg, ke)
    assert s2().device_status() == 0


def test_two_streams_at_once_and_refusals():
    b = _batch([(900, 3), (77, 1), (0, 9), (4000, 2)], 16, 4, 128, 64, None, 21)
    args = [b["q"].cuda(), b["kc"].cuda(), b["vc"].cuda(), i32(b["tab"]), i32([c for c, _ in b["lens"]]), i32(b["cu"])]
    want = s2().cache_attention(*args)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for st in streams * 4:
        with torch.cuda.stream(st):
            got.append(s2().cache_attention(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)
    f = s2().cache_attention
    with pytest.raises(ValueError, match="v_cache"):
        f(args[0], args[1], args[2][:-1], *args[3:])
    with pytest.raises(ValueError, match="contiguous"):
        f(args[0], args[1].transpose(1, 2).contiguous().transpose(1, 2), *args[2:])
    with pytest.raises(ValueError, match="int32"):
        f(*args[:3], args[3].long(), *args[4:])
    with pytest.raises(ValueError, match="cu_seqlens"):
        f(*args[:5], args[5][:-1])
    with pytest.raises(ValueError, match="mask"):
        f(*args, mask=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(s2().S2AttnError, match="WORKSPACE"):
        f(*args, workspace=torch.zeros(64, device="cuda"))
    with pytest.raises(s2().S2AttnError, match="UNSUPPORTED"):
        f(args[0], args[1].view(-1, 8, 4, 128), args[2].view(-1, 8, 4, 128), *args[3:])
    with pytest.raises(s2().S2AttnError, match="INVALID"):
        f(args[0][:0].contiguous(), *args[1:])
    with pytest.raises(s2().S2AttnError, match="INVALID"):
        s2().cache_plan(args[4], args[4], args[3], i32([1]), 16, 0)


def test_projection_to_attention_decodes_a_prompt():
    """NF4 projection, plan, append and attention of a prompt in one step agree
    with projection, rotation and dense attention."""
    H, Hkv, D, K, N = 4, 2, 64, 256, 128
    codes, sq, c2 = (t.cuda() for t in I.make_nf4_weights((H + 2 * Hkv) * D, K, seed=2))
    x = I.randn_bf16((1, N, K), 30).cuda()
    q, k, v = s2().nf4_qkv(x, codes, sq, c2, H, Hkv, D)
    tab = s2().rope_table(N, D, 1.0)
    dense = s2().dense_causal_attn(s2().rope_apply(q, tab), s2().rope_apply(k, tab), v)[0]
    blocks = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    p = s2().cache_plan(i32([0]), i32([N]), blocks, torch.randperm(8, device="cuda").int(), 16, N)
    kc = torch.empty(8, 16, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    qr = s2().cache_append(q[0], k[0], v[0], tab, p.positions, p.slots, kc, vc)
    o, _ = s2().cache_attention(qr, kc, vc, blocks, i32([0]), p.cu_seqlens)
    a, b = to64(o), to64(dense)
    assert np.all(np.abs(a - b) <= 2 * 2.0 ** -8 * np.abs(b) + 2 * (2.0 ** -8 + 2.0 ** -12) * np.abs(to64(v)).max())
