"""CPU checks of the oracles of the query/key norm and of decoding over a paged
cache (against differences, against the attention oracle, and by hand), and of
the refusals of their entry points (nothing is launched)."""
import numpy as np
import pytest
import torch

import oracle.cache_ref as cr
import oracle.qknorm_ref as qr
import oracle.rope_ref as rr
import oracle.s2_ref as ref
import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import _lib

P = 1 << 20  # a 16-byte aligned fake device address (never dereferenced)


def _table(n, D):
    a = rr.rope_angles(n, D, 1.0)
    return np.stack((np.cos(a), np.sin(a)), -1)


def test_norm_rope_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, dy, w = rng.standard_normal((1, 5, 2, 8)), rng.standard_normal((1, 5, 2, 8)), rng.standard_normal(8)
    tab, eps, h = _table(5, 8), 1e-3, 1e-5
    f = lambda x_, w_: (qr.norm_rope(x_, w_, tab, eps) * dy).sum()  # noqa: E731
    dx, dw, dx_abs, dw_abs = qr.norm_rope_bwd(x, w, tab, dy, eps)
    for idx in [(0, 0, 0, 0), (0, 2, 1, 3), (0, 4, 0, 7), (0, 3, 1, 4)]:
        e = np.zeros_like(x)
        e[idx] = h
        # central differences: error O(h^2) of third derivatives of order 10, rounding 1e-16 / h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[idx]) < 1e-7
    for i in range(8):
        e = np.zeros(8)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7
    assert (np.abs(dx) <= dx_abs + 1e-12).all() and (np.abs(dw) <= dw_abs + 1e-12).all()


def test_norm_rope_oracle_is_rope_of_a_unit_row():
    x = np.random.default_rng(1).standard_normal((2, 6, 3, 16))
    u = qr.norm(x, np.ones(16), 0.0)
    np.testing.assert_allclose((u * u).mean(-1), 1.0, atol=1e-12)
    np.testing.assert_allclose(qr.norm_rope(x, None, _table(6, 16), 0.0), rr.rope_rotate(x, 1.0), atol=1e-12)


def test_attention_oracle_is_dense_causal_attention():
    rng = np.random.default_rng(2)
    n, H, Hkv, D = 9, 4, 2, 8
    q, k, v = rng.standard_normal((1, n, H, D)), rng.standard_normal((1, n, Hkv, D)), rng.standard_normal((1, n, Hkv, D))
    o_ref, lse_ref = ref.s2_attention_fwd(q, k, v, n)
    for ctx in (0, 1, 5, 8):
        o, lse, _ = cr.attention(q[0, ctx:], k[0], v[0], ctx, cr.visible(n - ctx))
        np.testing.assert_allclose(o, o_ref[0, ctx:], atol=1e-12)
        np.testing.assert_allclose(lse, lse_ref[0][:, ctx:], atol=1e-12)


def test_plan_oracle_by_hand():
    # request 0: 3 tokens in block 7, one more fits; request 1: nothing yet, 5 tokens in two new blocks
    tab = [[7, -1], [-1, -1]]
    cu, pos, slots, mask, counts, out = cr.plan([3, 0], [1, 5], tab, [4, 2, 9], 4, 8, parents=[-1, -1, 0, 0, 1, 2, 0, 0])
    assert cu.tolist() == [0, 1, 6] and out.tolist() == [[7, -1], [4, 2]] and counts.tolist() == [2, 2, 6, 0]
    assert slots.tolist() == [31, 16, 17, 18, 19, 8, -1, -1]
    assert pos.tolist() == [3, 0, 1, 1, 2, 2, 0, 0]
    assert mask.tolist() == [1, 1, 3, 5, 11, 21, 0, 0]


def qk_fwd(q=P, k=P, w=P, tab=P, yq=P, yk=P, B=1, N=5, H=4, Hkv=2, D=128, eps=1e-6):
    return _lib.s2attn_qknorm_rope_fwd(q, k, w, w, tab, yq, yk, B, N, H, Hkv, D, 1, eps, None)


def qk_bwd(p=P, N=5, H=4, Hkv=2, D=128, eps=1e-6, ws=P, wsb=1 << 30):
    return _lib.s2attn_qknorm_rope_bwd(p, p, p, p, p, p, p, p, p, p, p, 1, N, H, Hkv, D, 0, eps, ws, wsb, None)


def append(p=P, wq=P, wk=P, pos=P, T=3, H=4, Hkv=2, D=64, rows=9, slots=64, eps=1e-6):
    return _lib.s2attn_cache_append(p, p, p, wq, wk, p, pos, p, p, p, p, T, H, Hkv, D, rows, slots, 1, eps, None)


def plan(p=P, free=P, par=None, mask=None, R=2, maxb=4, nf=3, bs=16, T=5):
    return _lib.s2attn_cache_plan(p, p, p, free, par, p, p, p, mask, p, R, maxb, nf, bs, T, None)


def attn(p=P, tab=P, mask=None, T=3, R=2, H=4, Hkv=2, D=64, nb=8, bs=16, maxb=4, ws=P, wsb=1 << 30):
    return _lib.s2attn_cache_attn(p, p, p, tab, p, p, mask, p, p, T, R, H, Hkv, D, nb, bs, maxb, ws, wsb, None)


INVALID, UNSUP, MISAL, WS = (_lib.S2ATTN_ERR_INVALID_ARG, _lib.S2ATTN_ERR_UNSUPPORTED, _lib.S2ATTN_ERR_MISALIGNED,
                             _lib.S2ATTN_ERR_WORKSPACE)


@pytest.mark.parametrize("fn,kw,status", [
    (qk_fwd, dict(q=None), INVALID), (qk_fwd, dict(N=0), INVALID), (qk_fwd, dict(B=-1), INVALID),
    (qk_fwd, dict(eps=0.0), INVALID), (qk_fwd, dict(eps=-1e-6), INVALID), (qk_fwd, dict(eps=float("nan")), INVALID),
    (qk_fwd, dict(eps=float("inf")), INVALID), (qk_fwd, dict(eps=1e-40), INVALID),
    (qk_fwd, dict(D=96), UNSUP), (qk_fwd, dict(N=1 << 30, H=4), UNSUP), (qk_fwd, dict(q=P + 8), MISAL),
    (qk_fwd, dict(tab=P + 4), MISAL), (qk_fwd, dict(yk=P + 2), MISAL),
    (qk_bwd, dict(p=None), INVALID), (qk_bwd, dict(D=32), UNSUP), (qk_bwd, dict(p=P + 8), MISAL),
    (qk_bwd, dict(ws=None), WS), (qk_bwd, dict(wsb=1024), WS), (qk_bwd, dict(ws=P + 8), WS),
    (append, dict(p=None), INVALID), (append, dict(wq=None), INVALID), (append, dict(T=0), INVALID),
    (append, dict(rows=0), INVALID), (append, dict(slots=0), INVALID), (append, dict(D=80), UNSUP),
    (append, dict(slots=1 << 31), UNSUP), (append, dict(p=P + 8), MISAL), (append, dict(pos=P + 2), MISAL),
    (plan, dict(p=None), INVALID), (plan, dict(R=0), INVALID), (plan, dict(T=0), INVALID), (plan, dict(bs=0), INVALID),
    (plan, dict(free=None), INVALID), (plan, dict(nf=-1), INVALID), (plan, dict(par=P), INVALID),
    (plan, dict(mask=P), INVALID), (plan, dict(R=1 << 20, maxb=1 << 12), UNSUP), (plan, dict(p=P + 2), MISAL),
    (plan, dict(par=P, mask=P + 4), MISAL),
    (attn, dict(p=None), INVALID), (attn, dict(T=0), INVALID), (attn, dict(R=0), INVALID), (attn, dict(maxb=0), INVALID),
    (attn, dict(H=4, Hkv=3), INVALID), (attn, dict(D=96), UNSUP), (attn, dict(bs=8), UNSUP), (attn, dict(bs=48), UNSUP),
    (attn, dict(bs=512), UNSUP), (attn, dict(H=258, Hkv=2), UNSUP), (attn, dict(nb=1 << 28, bs=16), UNSUP), (attn, dict(T=1 << 29), UNSUP),
    (attn, dict(p=P + 8), MISAL), (attn, dict(tab=P + 1), MISAL), (attn, dict(mask=P + 4), MISAL),
    (attn, dict(ws=None), WS), (attn, dict(wsb=100), WS), (attn, dict(ws=P + 8), WS),
])
def test_refusals_before_any_launch(fn, kw, status):
    assert fn(**kw) == status
    assert _lib.s2attn_last_launch_count() == 0


def test_workspace_sizes():
    assert _lib.s2attn_qknorm_rope_bwd_workspace_bytes(96) == 0
    assert _lib.s2attn_qknorm_rope_bwd_workspace_bytes(128) > 0
    assert _lib.s2attn_cache_attn_workspace_bytes(256) == 0
    assert 0 < _lib.s2attn_cache_attn_workspace_bytes(64) < _lib.s2attn_cache_attn_workspace_bytes(128)


def test_python_calls_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    w, tab = torch.ones(64), torch.zeros(4, 32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        s2.qknorm_rope_forward(x, x, w, w, tab)
    with pytest.raises(ValueError, match="q must be"):
        s2.qknorm_rope_forward(x[0], x, w, w, tab)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        s2.cache_plan(i, i, torch.zeros(2, 3, dtype=torch.int32), i, 16, 4)
    with pytest.raises(ValueError, match="ctx_lens"):
        s2.cache_plan([1, 2], i, i, i, 16, 4)
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        s2.cache_attention(x, x, x, i, i, i)
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        s2.cache_append(x, x, x, tab, i, i, x, x)
    with pytest.raises(ValueError, match="CUDA"):  # the first operand names the device of the others
        s2.nf4_dequantize(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, dtype=torch.int8), torch.zeros(1))
    with pytest.raises(TypeError, match="torch.Tensor"):
        s2.api._need("x", 5, (1,))
