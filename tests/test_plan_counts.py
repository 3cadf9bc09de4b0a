"""What a caller does with the counts of cache_plan: it drops the first
counts[0] blocks of the free list, so these and no others must be in the tables
-- also where the token arrays end before the tokens do."""
import numpy as np
import pytest
import torch

import oracle.cache_ref as cr

# ctx, new, block size, table width, free blocks, places for tokens
CASES = [
    ([3, 0], [1, 5], 4, 2, 3, 8), ([3, 0], [1, 5], 4, 2, 3, 6), ([3, 0], [1, 5], 4, 2, 3, 5), ([3, 0], [1, 5], 4, 2, 3, 1),
    ([4, 8, 0], [4, 4, 9], 4, 3, 9, 4), ([4, 8, 0], [4, 4, 9], 4, 3, 9, 5), ([4, 8, 0], [4, 4, 9], 4, 3, 9, 13),
    ([4, 8, 0], [4, 4, 9], 4, 3, 1, 9), ([0] * 40, [7] * 40, 16, 2, 64, 100), ([15] * 300, [2] * 300, 16, 2, 250, 333),
    ([100, 3], [50, 50], 8, 13, 40, 60), ([0], [1000], 16, 70, 70, 1), ([0] * 1100, [1] * 1100, 1, 1, 2000, 1050),
    ([0] * 1100, [1] * 1100, 1, 1, 2000, 1024), ([0] * 1100, [1] * 1100, 1, 1, 2000, 1100), ([0] * 300, [1] * 300, 1, 1, 9, 256),
    ([5] * 1024 + [0] * 7, [1] * 1024 + [9] * 7, 4, 3, 3000, 1024), ([90] * 9, [40] * 9, 8, 12, 60, 100),
]


def _tables(ctx, bs, width, free):
    tab, at = np.full((len(ctx), width), -1), 10 ** 4
    for r, c in enumerate(ctx):
        n = min(-(-c // bs), width)
        tab[r, :n] = np.arange(at, at + n)
        at += n
    return tab, np.arange(free)[::-1] + 7


def _check(tab, free, counts, out, total):
    new = out[(tab < 0) & (out >= 0)]
    assert counts[0] == len(new) and set(new) == set(free[:counts[0]]), (counts, new)
    assert np.array_equal(out[tab >= 0], tab[tab >= 0]) and counts[2] == total


@pytest.mark.parametrize("ctx,new,bs,width,nf,T", CASES)
def test_blocks_taken_are_those_in_the_tables_of_the_oracle(ctx, new, bs, width, nf, T):
    tab, free = _tables(ctx, bs, width, nf)
    _, _, slots, _, counts, out = cr.plan(ctx, new, tab, free, bs, T)
    _check(tab, free, counts, out, sum(new))
    assert all(s // bs in out for s in slots[slots >= 0])


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,new,bs,width,nf,T", CASES)
def test_blocks_taken_are_those_in_the_tables(ctx, new, bs, width, nf, T):
    import sparse_attention_attn_b200 as s2
    tab, free = _tables(ctx, bs, width, nf)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    d_tab = i32(tab)
    p = s2.cache_plan(i32(ctx), i32(new), d_tab, i32(free), bs, T)
    want = cr.plan(ctx, new, tab, free, bs, T)
    for got, ref in zip((p.cu_seqlens, p.positions, p.slots, p.counts, d_tab), (*want[:3], *want[4:]), strict=True):
        assert np.array_equal(got.cpu().numpy(), ref)
    _check(tab, free, p.counts.tolist(), d_tab.cpu().numpy(), sum(new))
