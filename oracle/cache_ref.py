"""fp64 / integer oracle of decoding over a paged cache: block planning, the
ancestor masks of drafted trees, and attention of new tokens over cached keys.
Written from the definitions with plain loops; nothing of the library is used.
"""
import numpy as np


def plan(ctx_lens, new_lens, block_tables, free_blocks, block_size, num_tokens, parents=None):
    """(cu_seqlens, positions, slots, mask, counts, block_tables) as arrays."""
    tab = np.array(block_tables, dtype=np.int64)
    width, bs, T = tab.shape[1], block_size, num_tokens
    cu = [0]
    pos, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    mask = np.zeros(T, np.uint64)
    wanted = taken = lost = 0
    for i, (ctx, new) in enumerate(zip(ctx_lens, new_lens)):
        ctx, new = max(int(ctx), 0), max(int(new), 0)
        have = min(-(-ctx // bs), width)
        need = min(-(-(ctx + new) // bs), width)
        opened = {}
        for b in range(have, need):
            opened[b] = int(free_blocks[wanted]) if wanted < len(free_blocks) else -1
            wanted += 1
        for j in range(new):
            t, p = cu[-1] + j, ctx + j
            b = p // bs
            blk = -1 if b >= width else (opened[b] if b in opened else int(tab[i, b]))
            if b >= width or (b in opened and blk < 0):
                lost += 1
            if t >= T:
                continue
            if b in opened and p % bs == 0:
                tab[i, b] = blk
                taken += blk >= 0  # a block is taken when a table names it
            if blk >= 0:
                slots[t] = blk * bs + p % bs
            depth, bits = j, 0
            if parents is not None:
                depth, at = 0, j
                bits = 1 << j if j < 64 else 0
                while True:
                    up = int(parents[cu[-1] + at])
                    if up < 0 or up >= at:
                        break
                    bits |= 1 << up if up < 64 else 0
                    depth, at = depth + 1, up
            mask[t] = np.uint64(bits)
            pos[t] = ctx + depth
        cu.append(cu[-1] + new)
    counts = [taken, wanted, cu[-1], lost]
    return np.array(cu), pos, slots, mask.view(np.int64), np.array(counts), tab


def visible(n, mask=None):
    """[n, n] truth values: does new token j see new token i of its request."""
    j = np.arange(n)
    if mask is None:
        return j[None, :] <= j[:, None]
    out = np.zeros((n, n), bool)
    for t in range(n):
        bits = int(mask[t]) & (2 ** 64 - 1)
        for i in range(min(n, 64)):
            out[t, i] = bits >> i & 1 == 1
    return out


def attention(q, k, v, ctx, see):
    """One request: q [n, H, D] over k, v [ctx + n, Hkv, D]; see [n, n].
    Returns o, lse [H, n] and the weighted mean of |v| (the rounding of the
    weights to bf16 moves o by at most 2^-8 of it).  Keys a row does not see
    are left out, whatever they hold."""
    n, H, D = q.shape
    rep = H // k.shape[1]
    o, lse, mag = np.zeros((n, H, D)), np.full((H, n), -np.inf), np.zeros((n, H, D))
    for j in range(n):
        keys = np.concatenate((np.arange(ctx), ctx + np.nonzero(see[j])[0]))
        if len(keys) == 0:
            continue
        for h in range(H):
            s = k[keys, h // rep] @ q[j, h] / np.sqrt(D)
            m = s.max()
            e = np.exp(s - m)
            lse[h, j] = m + np.log(e.sum())
            p = e / e.sum()
            o[j, h] = p @ v[keys, h // rep]
            mag[j, h] = p @ np.abs(v[keys, h // rep])
    return o, lse, mag
