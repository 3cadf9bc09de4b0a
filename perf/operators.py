"""The cached-decoding and query/key-norm operators, as cases with inputs, a plain form, and a 64-bit definition.

Operators (an "op" of a case):

* ``norm_fwd`` / ``norm_bwd``: root-mean-square norm of every query and key head with a learned weight, and the
  rotation by position in the same pass (training layout [B, N, heads, D]); the backward gives the gradients of
  q, k and of both weights;
* ``append``: the same norm (or none) and rotation for the new tokens of a ragged batch, whose rotated keys and
  values go into a paged cache at given slots (serving layout [T, heads, D]);
* ``plan``: blocks of the cache for the new tokens of every request, their slots, positions and (for a tree of
  drafted tokens) the mask of their ancestors, built on the GPU from the requests' lengths;
* ``attend``: attention of new tokens -- one, a chain or a tree of drafts per request -- over the paged cache.

``run`` computes the plain form in elementary torch operations; with ``own`` set it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BASE = 10000.0
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the tiny workload's layer (4 heads of 64, 1024 tokens): a small model's step, where launch latency counts
        dict(name="norm-fwd-tiny", op="norm_fwd", B=1, N=1024, H=4, Hkv=4, D=64, w="fp32"),
        # a Qwen3-8B layer (grouped queries, normed heads) at 16K tokens: the forward of a training step
        dict(name="norm-fwd-qwen3-8b", op="norm_fwd", B=1, N=16384, H=32, Hkv=8, D=128, w="bf16"),
        # two short sequences of odd length, three query heads to a key head: fine-tuning on short texts
        dict(name="norm-bwd-odd", op="norm_bwd", B=2, N=1537, H=6, Hkv=2, D=64, w="fp32"),
        # the LLaMA2-70B layer's head layout at 32K tokens: the largest backward of a training step
        dict(name="norm-bwd-64h-32k", op="norm_bwd", B=1, N=32768, H=64, Hkv=8, D=128, w="bf16"),
        # one token for each of 8 running requests: the step between projection and attention when decoding
        dict(name="append-decode", op="append", R=8, new_lo=1, new_hi=1, ctx=2000, H=32, Hkv=8, D=128, bs=16,
             norm=True, pad=0),
        # prompts of up to 4K tokens entering the cache, rotation only (a LLaMA2-7B layer), padded to a fixed size
        dict(name="append-prefill", op="append", R=7, new_lo=301, new_hi=4095, ctx=0, H=32, Hkv=32, D=128, bs=64,
             norm=False, pad=61),
        # block bookkeeping of 64 decoding requests, once per generated token: pure latency
        dict(name="plan-decode", op="plan", R=64, new_lo=1, new_hi=1, ctx=8191, bs=16, tree=False, pad=0),
        # 1024 requests with trees of up to 64 drafts each: the bookkeeping of a large speculative batch
        dict(name="plan-tree", op="plan", R=1024, new_lo=17, new_hi=64, ctx=16384, bs=32, tree=True, pad=100),
        # a single chat at 4K tokens, one token at a time: the smallest call
        dict(name="attend-one", op="attend", R=1, ctx_lo=4097, ctx_hi=4097, new_lo=1, new_hi=1, H=32, Hkv=8, D=128,
             bs=16, tree=False),
        # 64 running requests of very different lengths, one token each (Qwen3-8B heads): ordinary batched decoding
        dict(name="attend-batch", op="attend", R=64, ctx_lo=333, ctx_hi=16384, new_lo=1, new_hi=1, H=32, Hkv=8,
             D=128, bs=64, tree=False),
        # trees of about 60 drafts over 8K-token contexts, 8 query heads to a key head: verification of drafts
        dict(name="attend-tree", op="attend", R=16, ctx_lo=4001, ctx_hi=12289, new_lo=57, new_hi=64, H=64, Hkv=8,
             D=128, bs=32, tree=True),
        # one request at the 100K-token context, every head with its own keys, a chain of 5 drafts
        dict(name="attend-long", op="attend", R=1, ctx_lo=102400, ctx_hi=102400, new_lo=5, new_hi=5, H=32, Hkv=32,
             D=128, bs=128, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(4, 4), (32, 32), (32, 8), (64, 8), (6, 2), (8, 1), (12, 4)])


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "append", "plan", "attend", "attend"])
    D = rng.choice([64, 128, 128])
    bs = rng.choice([16, 32, 64, 128, 256])
    H, Hkv = _heads(rng)
    if op in ("norm_fwd", "norm_bwd"):
        B, N = rng.choice([1, 1, 2, 3]), _log(rng, 1, 32768)
        N = max(1, min(N, 32768 * 72 // (B * (H + Hkv))))
        return dict(op=op, B=B, N=N, H=H, Hkv=Hkv, D=D, w=rng.choice(["fp32", "bf16"]))
    if op == "append":
        R = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, 15000 // R))
        return dict(op=op, R=R, new_lo=rng.randint(1, hi), new_hi=hi, ctx=_log(rng, 1, max(2, 60000 // R)), H=H,
                    Hkv=Hkv, D=D, bs=bs, norm=rng.random() < 0.6, pad=rng.choice([0, 0, rng.randint(1, 99)]))
    if op == "plan":
        R, tree = _log(rng, 1, 1024), rng.random() < 0.5
        hi = _log(rng, 1, 64 if tree else max(1, 60000 // R))
        return dict(op=op, R=R, new_lo=rng.randint(0, hi), new_hi=hi, ctx=_log(rng, 1, 16384), bs=bs, tree=tree,
                    pad=rng.choice([0, rng.randint(1, 300)]))
    R, ctx = _log(rng, 1, 64), _log(rng, 1, 65536)
    ctx = max(1, min(ctx, 4_000_000 // (R * Hkv)))
    kind = rng.choice(["one", "chain", "tree"])
    hi = 1 if kind == "one" else _log(rng, 2, 64 if kind == "tree" else 200)
    hi = max(1, min(hi, int(2.2e11 / (R * (ctx + hi) * H * 4 * D))))
    return dict(op="attend", R=R, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx, new_lo=rng.randint(1, hi), new_hi=hi, H=H,
                Hkv=Hkv, D=D, bs=bs, tree=kind == "tree" and hi > 1)


def _spread(lo, hi, n, phase=0.5):
    """n whole numbers over [lo, hi], well spread and the same for every seed (the work is the case's alone)."""
    return [lo + int(((i + 1) * GOLDEN + phase) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(c):
    new = _spread(c["new_lo"], c["new_hi"], c["R"])
    if c["op"] == "attend":
        ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["R"], 0.25)
    else:
        ctx = _spread(0, c["ctx"], c["R"], 0.25)
    return ctx, new


# ------------------------------------------------------------------ inputs

def _rope_table(n, D):
    i = torch.arange(D // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * torch.exp(-2.0 * i / D * math.log(BASE))
    return torch.stack((torch.cos(a), torch.sin(a)), -1).to(torch.float32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    hg = np.random.default_rng(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def weight(D, kind):
        w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
        return w.to(torch.bfloat16) if kind == "bf16" else w

    def ints(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")

    s = {"op": c["op"], "case": c}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        B, N, H, Hkv, D = c["B"], c["N"], c["H"], c["Hkv"], c["D"]
        s.update(q=randn(B, N, H, D), k=randn(B, N, Hkv, D), w_q=weight(D, c["w"]), w_k=weight(D, c["w"]),
                 table=_rope_table(N, D))
        if c["op"] == "norm_bwd":
            s.update(dq=randn(B, N, H, D), dk=randn(B, N, Hkv, D))
        return s

    ctx, new = _lens(c)
    order = hg.permutation(c["R"])
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    bs, R = c["bs"], c["R"]
    have = [-(-x // bs) for x in ctx]
    total = [-(-(x + n) // bs) for x, n in zip(ctx, new)]
    pad = c.get("pad", 0)
    cu = np.concatenate(([0], np.cumsum(new))).astype(np.int64)
    T = max(1, int(cu[-1]) + pad)
    s.update(ctx_host=ctx, new_host=new, bs=bs, T=T)
    parents = None
    if c.get("tree"):  # every draft hangs on one of the few before it, or on the context
        parents = np.full(T, -1, np.int64)
        for r in range(R):
            j = np.arange(new[r])
            parents[cu[r]:cu[r + 1]] = np.maximum(-1, j - hg.integers(1, 9, new[r]))
        s["parents_host"] = parents
    if c["op"] == "plan":
        nb = sum(total) + 8
        ids = hg.permutation(nb)
        tab = np.full((R, max(1, max(total)) + 1), -1, np.int64)
        at = 0
        for r in range(R):
            tab[r, :have[r]] = ids[at:at + have[r]]
            at += have[r]
        s.update(ctx_lens=ints(ctx), new_lens=ints(new), block_tables=ints(tab), free_blocks=ints(ids[at:]),
                 parents=None if parents is None else ints(parents))
        return s

    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    nb = sum(total) + 4
    ids = hg.permutation(nb)
    tab = np.full((R, max(1, max(total))), -1, np.int64)
    pos, slot, at = np.zeros(T, np.int64), np.full(T, -1, np.int64), 0
    for r in range(R):
        tab[r, :total[r]] = ids[at:at + total[r]]
        at += total[r]
        p = ctx[r] + np.arange(new[r])
        pos[cu[r]:cu[r + 1]] = p
        slot[cu[r]:cu[r + 1]] = tab[r, p // bs] * bs + p % bs
    s.update(k_cache=randn(nb, bs, Hkv, D), v_cache=randn(nb, bs, Hkv, D), q=randn(T, H, D))
    if c["op"] == "append":
        s.update(k=randn(T, Hkv, D), v=randn(T, Hkv, D), positions=ints(pos), slots=ints(slot),
                 table=_rope_table(max(max(x + n for x, n in zip(ctx, new)), 1), D),
                 w_q=weight(D, "bf16") if c["norm"] else None, w_k=weight(D, "bf16") if c["norm"] else None,
                 q_out=torch.zeros(T, H, D, device="cuda", dtype=torch.bfloat16))
        return s
    mask = None
    if parents is not None:
        mask = np.zeros(T, np.uint64)
        for r in range(R):
            m = mask[cu[r]:cu[r + 1]]
            for j in range(new[r]):
                up = parents[cu[r] + j]
                m[j] = np.uint64(1 << j) | (m[up] if up >= 0 else np.uint64(0))
        mask = torch.from_numpy(mask.view(np.int64)).cuda()
    s.update(block_tables=ints(tab), ctx_lens=ints(ctx), cu_seqlens=ints(cu), mask=mask)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import sparse_attention_attn_b200 as s2
    if s["op"] == "norm_fwd":
        return s2.qknorm_rope_forward(s["q"], s["k"], s["w_q"], s["w_k"], s["table"], eps=EPS)
    if s["op"] == "norm_bwd":
        return s2.qknorm_rope_backward(s["q"], s["k"], s["w_q"], s["w_k"], s["dq"], s["dk"], s["table"], eps=EPS)
    if s["op"] == "append":
        q = s2.cache_append(s["q"], s["k"], s["v"], s["table"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                            w_q=s["w_q"], w_k=s["w_k"], eps=EPS, q_out=s["q_out"])
        return q, s["k_cache"], s["v_cache"]
    if s["op"] == "plan":
        p = s2.cache_plan(s["ctx_lens"], s["new_lens"], s["block_tables"], s["free_blocks"], s["bs"], s["T"],
                          parents=s["parents"])
        out = [p.cu_seqlens, p.positions, p.slots, p.counts, s["block_tables"]]
        return out + [p.mask] if s["parents"] is not None else out
    return s2.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["ctx_lens"], s["cu_seqlens"],
                              mask=s["mask"])


def _norm_rope(x, w, cos, sin):
    """x [..., D] in 32 bits, cos and sin broadcast against [..., D/2]; w None: no norm."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _norm_rope_bwd(x, w, dy, cos, sin):
    x, dy = x.float(), dy.float()
    a, b = dy.chunk(2, -1)
    du = torch.cat((a * cos + b * sin, b * cos - a * sin), -1)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xn = x * r
    dw = (du * xn).sum((0, 1, 2), dtype=torch.float64)  # a long sum
    g = du * w.float()
    dx = r * (g - xn * (g * xn).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw.to(w.dtype)


def _run_plain(s):
    if s["op"] in ("norm_fwd", "norm_bwd"):
        cos, sin = (s["table"][None, :, None, :, i] for i in (0, 1))
        if s["op"] == "norm_fwd":
            return tuple(_norm_rope(s[x].float(), s["w_" + x], cos, sin).to(torch.bfloat16) for x in ("q", "k"))
        dq, dwq = _norm_rope_bwd(s["q"], s["w_q"], s["dq"], cos, sin)
        dk, dwk = _norm_rope_bwd(s["k"], s["w_k"], s["dk"], cos, sin)
        return dq, dk, dwq, dwk
    if s["op"] == "append":
        t = sum(s["new_host"])
        tab = s["table"][s["positions"][:t].long()]
        cos, sin = tab[:, None, :, 0], tab[:, None, :, 1]
        at = s["slots"][:t].long()
        s["q_out"][:t] = _norm_rope(s["q"][:t].float(), s["w_q"], cos, sin).to(torch.bfloat16)
        kc, vc = s["k_cache"], s["v_cache"]
        kc.view(-1, *kc.shape[2:])[at] = _norm_rope(s["k"][:t].float(), s["w_k"], cos, sin).to(torch.bfloat16)
        vc.view(-1, *vc.shape[2:])[at] = s["v"][:t]
        return s["q_out"], kc, vc
    if s["op"] == "plan":
        return _plan_plain(s)
    return _attend_plain(s)


def _plan_plain(s):
    ctx, new, bs, T = s["ctx_lens"].long(), s["new_lens"].long(), s["bs"], s["T"]
    dev, R = ctx.device, ctx.numel()
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)))
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    real = r < R
    rr = r.clamp(max=R - 1)
    j = t - cu[rr]
    place = ctx[rr] + j  # where the token lies in its request
    have, need = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    first = torch.cat((torch.zeros(1, dtype=torch.long, device=dev), (need - have).cumsum(0)))
    col = torch.arange(s["block_tables"].shape[1], device=dev)[None]
    mine = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:-1, None] + col - have[:, None]).clamp(0, s["free_blocks"].numel() - 1)
    tab = torch.where(mine, s["free_blocks"].long()[at], s["block_tables"].long())
    s["block_tables"].copy_(tab)
    blk = tab[rr, (place // bs).clamp(max=tab.shape[1] - 1)]
    slots = torch.where(real, blk * bs + place % bs, -1)
    depth, mask = j, None
    if s["parents"] is not None:  # climb from every draft to the root at once
        up, depth = s["parents"].long(), torch.zeros_like(t)
        mask = torch.where(real, torch.ones_like(t) << j.clamp(0, 63), 0)
        live = torch.where(real, up, -1)
        for _ in range(64):
            on = live >= 0
            depth = depth + on
            mask = mask | torch.where(on, torch.ones_like(t) << live.clamp(min=0), 0)
            live = torch.where(on, up[(cu[rr] + live.clamp(min=0)).clamp(max=T - 1)], -1)
    pos = torch.where(real, ctx[rr] + depth, 0)
    counts = torch.stack((first[-1], first[-1], cu[-1], torch.zeros_like(cu[-1])))
    out = [cu.int(), pos.int(), slots.int(), counts.int(), s["block_tables"]]
    return out + [mask] if mask is not None else out


def _attend_plain(s):
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, H, D = q.shape
    Hkv = kc.shape[2]
    rep, bs, scale = H // Hkv, s["bs"], 1.0 / math.sqrt(D)
    o = torch.empty_like(q)
    lse = torch.empty(H, T, dtype=torch.float32, device=q.device)
    t0 = 0
    for r, (ctx, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        L = ctx + n
        blocks = s["block_tables"][r, :-(-L // bs)].long()
        k = kc[blocks].reshape(-1, Hkv, D)[:L].float().permute(1, 2, 0)  # [Hkv, D, L]
        v = vc[blocks].reshape(-1, Hkv, D)[:L].float().permute(1, 0, 2)
        qr = q[t0:t0 + n].float().view(n, Hkv, rep, D).permute(1, 0, 2, 3).reshape(Hkv, n * rep, D)
        x = torch.matmul(qr, k).view(Hkv, n, rep, L) * scale
        j = torch.arange(n, device=q.device)
        if s["mask"] is None:
            see = j[None, :] <= j[:, None]
        else:
            see = (s["mask"][t0:t0 + n, None] >> j[None, :]) & 1 == 1
        x[..., ctx:] = x[..., ctx:].masked_fill(~see[None, :, None, :], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(-1, keepdim=True)
        out = torch.matmul(p.view(Hkv, n * rep, L), v).view(Hkv, n, rep, D) / z
        o[t0:t0 + n] = out.permute(1, 0, 2, 3).reshape(n, H, D).to(o.dtype)
        lse[:, t0:t0 + n] = (m + torch.log(z))[..., 0].permute(0, 2, 1).reshape(H, n)
        t0 += n
    return o, lse


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: t.double()  # noqa: E731
    if s["op"] in ("norm_fwd", "norm_bwd"):
        out, grads_w = [], []
        for x, w, dy in (("q", "w_q", "dq"), ("k", "w_k", "dk")):
            heads = []
            dw = torch.zeros(s["case"]["D"], dtype=torch.float64, device="cuda")
            c, sn = f(s["table"][..., 0]), f(s["table"][..., 1])
            half = s["case"]["D"] // 2
            for h in range(s[x].shape[2]):  # one head at a time: a rotation is the product with e^{ia}
                xh = f(s[x][:, :, h])
                rms = torch.sqrt((xh ** 2).sum(-1, keepdim=True) / (2 * half) + EPS)
                turn = torch.complex(c, sn)[None]
                if s["op"] == "norm_fwd":
                    u = xh / rms * f(s[w])
                    z = torch.complex(u[..., :half].contiguous(), u[..., half:].contiguous()) * turn
                    heads.append(torch.cat((z.real, z.imag), -1))
                else:
                    d = f(s[dy][:, :, h])
                    z = torch.complex(d[..., :half].contiguous(), d[..., half:].contiguous()) * turn.conj()
                    du = torch.cat((z.real, z.imag), -1)
                    dw += (du * xh / rms).sum((0, 1))
                    gg = du * f(s[w])
                    heads.append(gg / rms - xh * (gg * xh).sum(-1, keepdim=True) / (2 * half * rms ** 3))
            out.append(torch.stack(heads, 2))
            grads_w.append(dw)
        return tuple(out) if s["op"] == "norm_fwd" else tuple(out + grads_w)
    if s["op"] == "append":
        t = sum(s["new_host"])
        tab = f(s["table"])[s["positions"][:t].long()]
        res = []
        for x, w in (("q", "w_q"), ("k", "w_k")):
            v = f(s[x][:t])
            if s[w] is not None:
                v = v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + EPS) * f(s[w])
            half = v.shape[-1] // 2
            z = torch.complex(v[..., :half].contiguous(), v[..., half:].contiguous())
            z = z * torch.complex(tab[..., 0].contiguous(), tab[..., 1].contiguous())[:, None]
            res.append(torch.cat((z.real, z.imag), -1))
        q_out, kc, vc = f(s["q_out"]), f(s["k_cache"]), f(s["v_cache"])
        q_out[:t] = res[0]
        blk, off = s["slots"][:t].long() // s["bs"], s["slots"][:t].long() % s["bs"]
        kc[blk, off] = res[1]
        vc[blk, off] = f(s["v"][:t])
        return q_out, kc, vc
    if s["op"] == "plan":
        return _plan_exact(s)
    q, T, H = s["q"], s["q"].shape[0], s["q"].shape[1]
    D, Hkv, bs = q.shape[2], s["k_cache"].shape[2], s["bs"]
    o = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(H, T, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (ctx, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        at = torch.arange(ctx + n, device="cuda")
        blk = s["block_tables"][r].long()[at // bs]
        see = torch.ones(n, ctx + n, dtype=torch.bool, device="cuda")
        for j in range(n):
            if s["mask"] is None:
                see[j, ctx + j + 1:] = False
            else:
                bits = int(s["mask"][t0 + j]) & (2 ** 64 - 1)
                see[j, ctx:] = torch.tensor([bits >> i & 1 == 1 for i in range(n)], device="cuda")
        for g in range(Hkv):
            k, v = f(s["k_cache"][blk, at % bs, g]), f(s["v_cache"][blk, at % bs, g])
            hs = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            x = torch.einsum("nhd,ld->hnl", f(q[t0:t0 + n, hs]), k) / math.sqrt(D)
            x = torch.where(see[None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[hs, t0:t0 + n] = z
            o[t0:t0 + n, hs] = torch.einsum("hnl,ld->nhd", torch.exp(x - z[..., None]), v)
        t0 += n
    return o, lse


def _plan_exact(s):
    bs, T, R = s["bs"], s["T"], len(s["ctx_host"])
    tab, free = s["block_tables"].cpu().numpy().copy(), s["free_blocks"].cpu().numpy()
    cu, pos, slot = np.zeros(R + 1, np.int64), np.zeros(T, np.int64), np.full(T, -1, np.int64)
    mask, used, t = np.zeros(T, np.uint64), 0, 0
    for r, (ctx, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        for b in range(-(-ctx // bs), -(-(ctx + n) // bs)):
            tab[r, b] = free[used]
            used += 1
        for j in range(n):
            at, d = ctx + j, j
            slot[t] = int(tab[r, at // bs]) * bs + at % bs
            if "parents_host" in s:
                bits, d, up = 1 << j, 0, int(s["parents_host"][cu[r] + j])
                while up >= 0:
                    bits, d, up = bits | 1 << up, d + 1, int(s["parents_host"][cu[r] + up])
                mask[t] = np.uint64(bits)
            pos[t] = ctx + d
            t += 1
        cu[r + 1] = t
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    out = [i32(cu), i32(pos), i32(slot), i32([used, used, t, 0]), i32(tab)]
    return out + [torch.from_numpy(mask.view(np.int64)).cuda()] if "parents_host" in s else out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("norm_fwd", "norm_bwd"):
        rows, D = c["B"] * c["N"] * (c["H"] + c["Hkv"]), c["D"]
        w = 2 * D * (4 if c["w"] == "fp32" else 2)
        table = c["N"] * D * 4
        if c["op"] == "norm_fwd":
            return {"bytes": rows * D * 4 + table + w, "flops": rows * D * 7}
        return {"bytes": rows * D * 6 + table + 2 * w, "flops": rows * D * 14}
    ctx, new = _lens(c)
    t, L, bs = sum(new), sum(ctx) + sum(new), c["bs"]
    if c["op"] == "append":
        H, Hkv, D = c["H"], c["Hkv"], c["D"]
        return {"bytes": t * ((2 * H + 4 * Hkv) * D * 2 + D * 4 + 8), "flops": t * (H + Hkv) * D * (7 if c["norm"] else 3)}
    blocks = sum(-(-(x + n) // bs) for x, n in zip(ctx, new))
    if c["op"] == "plan":
        fresh = blocks - sum(-(-x // bs) for x in ctx)
        T = max(1, t + c["pad"])
        return {"bytes": 12 * c["R"] + 8 * fresh + 8 * T + (12 * T if c["tree"] else 0), "flops": 4 * T}
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    seen = sum(n * x + (n if c["tree"] else n * (n + 1) // 2) for x, n in zip(ctx, new))
    return {"bytes": L * Hkv * D * 4 + t * H * (D * 4 + 4) + 4 * blocks + 8 * c["R"], "flops": 4 * D * H * seen}
