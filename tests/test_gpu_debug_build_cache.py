"""The debug build on the norm and decoding calls: on valid calls no index check
fires and the outputs have the same bits as the default build's, in both
attention kernels and in clusters.  A block number outside the cache is
recorded by both.  Each build runs in its own process."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_attn_b200", "csrc")

SCRIPT = r'''
import hashlib, json, sys
import torch
sys.path.insert(0, sys.argv[1])
import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import _lib, inputs as I
dev = torch.device("cuda:0")
out = {"debug": _lib.load().s2attn_debug_checks()}
h = lambda *ts: hashlib.sha256(b"".join(t.detach().cpu().contiguous().view(torch.uint8).numpy().tobytes() for t in ts)).hexdigest()
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
def done(name, *ts):
    torch.cuda.synchronize()
    out[name] = [h(*ts), s2.device_status()]
for B, N, H, Hkv, D in ((1, 1, 1, 1, 64), (2, 333, 7, 3, 128), (1, 9000, 8, 8, 64)):
    q, k, gq, gk = (I.randn_bf16((B, N, n, D), i).to(dev) for i, n in enumerate((H, Hkv, H, Hkv)))
    w, tab = torch.linspace(0.5, 1.5, D, device=dev), s2.rope_table(N, D, 1.0)
    done(f"norm {N}", *s2.qknorm_rope_forward(q, k, w, w, tab), *s2.qknorm_rope_backward(q, k, w, w, gq, gk, tab))
ctx, new = [37, 0, 700, 5, 64, 1000, 3], [3, 5, 1, 0, 64, 70, 200]
R, T, bs, width = len(ctx), sum(new) + 5, 16, 80
par = [max(-1, j - 1 - (j * 7) % 5) for n in new for j in range(n)] + [-1] * 5
for H, Hkv, D in ((8, 2, 128), (6, 6, 64), (40, 1, 64)):
    q, k, v = (I.randn_bf16((T, n, D), 7 + i).to(dev) for i, n in enumerate((H, Hkv, Hkv)))
    kc, vc = I.randn_bf16((300, bs, Hkv, D), 11).to(dev), I.randn_bf16((300, bs, Hkv, D), 12).to(dev)
    rope = s2.rope_table(2048, D, 1.0)
    blocks = torch.full((R, width), -1, dtype=torch.int32)
    at = 0
    for r, c in enumerate(ctx):
        n = -(-c // bs)
        blocks[r, :n], at = torch.arange(at, at + n), at + n
    free = at + torch.randperm(300 - at, generator=torch.Generator().manual_seed(1)).int()
    for tree in (False, True):
        t = blocks.to(dev)
        p = s2.cache_plan(i32(ctx), i32(new), t, free.to(dev), bs, T,
                          i32(par) if tree else None)
        done(f"plan {H} {tree}", p.cu_seqlens, p.positions, p.slots, p.counts, t, *([p.mask] if tree else []))
        k2, v2 = kc.clone(), vc.clone()
        qq = s2.cache_append(q, k, v, rope, p.positions, p.slots, k2, v2, q_out=torch.zeros_like(q))
        done(f"append {H} {tree}", qq, k2, v2)
        for kern in ("dec", "cluster", "tc"):
            _lib.s2attn_set_tile_override("cache=" + kern)
            o, l = s2.cache_attention(qq, k2, v2, t, i32(ctx), p.cu_seqlens, mask=p.mask, out=torch.zeros_like(q),
                                      lse=torch.zeros(H, T, device=dev))
            done(f"attn {H} {tree} {kern}", o, l)
        _lib.s2attn_set_tile_override(None)
t[2, 3] = 300
s2.cache_attention(qq, k2, v2, t, i32(ctx), p.cu_seqlens)
out["bad"] = s2.device_status()
print(json.dumps(out))
'''


def test_every_kernel_source_of_these_calls_has_index_checks():
    for f in ("s2_qknorm.cu", "s2_cache.cu", "s2_cache.cuh", "s2_cache_dec.cu", "s2_cache_tc.cu"):
        with open(os.path.join(CSRC, f)) as fh:
            assert "in_bounds(" in fh.read(), f


def _run(debug: bool):
    env = dict(os.environ)
    env.pop("S2ATTN_DEBUG", None)
    if debug:
        env["S2ATTN_DEBUG"] = "1"
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.gpu
def test_debug_build_agrees_and_no_check_fires():
    from sparse_attention_attn_b200 import build
    build.build(debug=True)
    rel, dbg = _run(False), _run(True)
    assert (rel.pop("debug"), dbg.pop("debug")) == (0, 1)
    assert rel.pop("bad") == dbg.pop("bad") == 7
    assert all(status == 0 for _, status in dbg.values()), {k: v[1] for k, v in dbg.items() if v[1]}
    assert rel == dbg
