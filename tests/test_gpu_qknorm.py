"""GPU parity of the query/key norm with rotation -- forward, backward, autograd
and the serving form that appends to a paged cache -- against the fp64 oracle.

Tolerances, elementwise.  A bf16 result is off by half a step, 2^-8 of its
value (2^-8 = finfo(bf16).eps / 2).  The fp32 arithmetic before it: y is a sum
of two products of u = r x w, each with at most about 8 roundings of 2^-24 and
the 2-ulp reciprocal square root, so 2^-20 of |u1| + |u2| covers it; dx is a
sum of the terms whose absolute values the oracle adds up (dx_abs), each with
fewer than 64 roundings (the row sums have 128 terms added in 16 + 3 steps):
2^-18 dx_abs.  dw adds one product per row: at most 48 rows in sequence per
thread in these shapes, then a tree: (48 + 40) 2^-24 < 2^-17 of the sum of
absolute terms; bf16 weights add 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import oracle.qknorm_ref as qr
from sparse_attention_attn_b200 import inputs as I
from tests.parity_util import check_grad, check_o, to64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def s2():
    import sparse_attention_attn_b200
    return sparse_attention_attn_b200


def _weights(D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.3 * torch.randn(D, generator=g)).to(dtype)


def _fwd_bound(x, w, table, ref):
    u = np.abs(qr.norm(x, w, EPS) if w is not None else x)
    a, b = np.split(u, 2, axis=-1)
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.concatenate((a + b, a + b), -1) + 1e-30


SHAPES = [  # B, N, H, Hkv, D: one token, odd lengths, heads that fill no group, many rows
    (1, 1, 1, 1, 64), (1, 1, 1, 1, 128), (2, 3, 5, 1, 128), (1, 129, 6, 2, 64), (3, 77, 7, 7, 128), (2, 1000, 32, 8, 128),
    (1, 1537, 4, 4, 64),
]


def _case(B, N, H, Hkv, D, dtype, seed=0):
    q, k = I.randn_bf16((B, N, H, D), seed), I.randn_bf16((B, N, Hkv, D), seed + 1)
    dq, dk = I.randn_bf16((B, N, H, D), seed + 2), I.randn_bf16((B, N, Hkv, D), seed + 3)
    q[0, 0, 0] = 0  # a row of zeros: eps alone under the root
    k[-1, -1] *= 300
    return q, k, _weights(D, dtype, seed + 4), _weights(D, dtype, seed + 5), dq, dk


@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,H,Hkv,D", SHAPES)
def test_forward_and_backward_against_oracle(B, N, H, Hkv, D, wt):
    q, k, wq, wk, gq, gk = _case(B, N, H, Hkv, D, wt)
    tab = s2().rope_table(N, D, 0.5)
    t64 = to64(tab)
    d = [t.cuda() for t in (q, k, wq, wk, gq, gk)]
    yq, yk = s2().qknorm_rope_forward(*d[:4], tab, eps=EPS)
    dq, dk, dwq, dwk = s2().qknorm_rope_backward(*d, tab, eps=EPS)
    torch.cuda.synchronize()
    for x, w, dy, y, dx, dw in ((q, wq, gq, yq, dq, dwq), (k, wk, gk, yk, dk, dwk)):
        ref = qr.norm_rope(to64(x), to64(w), t64, EPS)
        assert np.all(np.abs(to64(y) - ref) <= _fwd_bound(to64(x), to64(w), t64, ref))
        dx_ref, dw_ref, dx_abs, dw_abs = qr.norm_rope_bwd(to64(x), to64(w), t64, to64(dy), EPS)
        assert np.all(np.abs(to64(dx) - dx_ref) <= 2.0 ** -8 * np.abs(dx_ref) + 2.0 ** -18 * dx_abs)
        half = 2.0 ** -8 if wt == torch.bfloat16 else 2.0 ** -24
        assert dw.dtype == wt
        assert np.all(np.abs(to64(dw) - dw_ref) <= half * np.abs(dw_ref) + 2.0 ** -17 * dw_abs)


def test_in_place_and_repeat_give_the_same_bits():
    q, k, wq, wk, gq, gk = (t.cuda() for t in _case(2, 333, 6, 2, 128, torch.float32))
    tab = s2().rope_table(333, 128, 1.0)
    yq, yk = s2().qknorm_rope_forward(q, k, wq, wk, tab)
    first = s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab)
    again = s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab, dq=gq, dk=gk)  # over the incoming gradients
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    s2().qknorm_rope_forward(q, k, wq, wk, tab, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)


def test_non_finite_rows_stay_in_their_rows():
    q, k, wq, wk, _, _ = (t.cuda() for t in _case(1, 40, 4, 2, 64, torch.float32))
    tab = s2().rope_table(40, 64, 1.0)
    yq, yk = s2().qknorm_rope_forward(q, k, wq, wk, tab)
    q2 = q.clone()
    q2[0, 7, 1, 5], q2[0, 39, 3, 63] = float("nan"), float("inf")
    zq, zk = s2().qknorm_rope_forward(q2, k, wq, wk, tab)
    keep = torch.ones(40, 4, dtype=torch.bool)
    keep[7, 1] = keep[39, 3] = False
    assert torch.equal(zq[0][keep.cuda()], yq[0][keep.cuda()]) and torch.equal(zk, yk)
    assert torch.isnan(zq[0, 7, 1]).all() and not torch.isfinite(zq[0, 39, 3]).all()


def test_autograd_through_s2_attention():
    """s2_qknorm_attn (norm, rotation, shifted attention) against the oracle of
    each step in turn, and leaves used with broadcast gradients."""
    import oracle.s2_ref as ref
    B, N, H, Hkv, D, G = 1, 512, 4, 2, 64, 256
    q, k, wq, wk, do, _ = _case(B, N, H, Hkv, D, torch.float32, seed=40)
    v = I.randn_bf16((B, N, Hkv, D), 50)
    tab = s2().rope_table(N, D, 1.0)
    leaves = [t.cuda().requires_grad_() for t in (q, k, v, wq, wk)]
    o = s2().s2_qknorm_attn(*leaves, G, tab, EPS)
    o.backward(do.cuda())
    t64 = to64(tab)
    # the attention reads the rotated q, k rounded to bf16
    yq, yk = s2().qknorm_rope_forward(*(t.detach() for t in (leaves[0], leaves[1], leaves[3], leaves[4])), tab)
    check_o(to64(o), ref.s2_attention_fwd(to64(yq), to64(yk), to64(v), G)[0])
    gq, gk, gv, _ = ref.s2_attention_bwd(to64(yq), to64(yk), to64(v), to64(do), G)
    for leaf, x, w, wl, g in ((leaves[0], q, wq, leaves[3], gq), (leaves[1], k, wk, leaves[4], gk)):
        dx, dw, _, _ = qr.norm_rope_bwd(to64(x), to64(w), t64, g, EPS)
        # a row of zeros has r = 1/sqrt(eps) = 1000: its gradient is compared apart from the others
        got = to64(leaf.grad)
        zero = np.abs(to64(x)).sum(-1) == 0
        check_grad("dx", got[~zero], dx[~zero])
        if zero.any():
            check_grad("dx of zero rows", got[zero], dx[zero])
        check_grad("dw", to64(wl.grad), dw)
    check_grad("dv", to64(leaves[2].grad), gv)
    # a broadcast (stride 0) incoming gradient
    a, b = s2().QKNormRope.apply(leaves[0], leaves[1], leaves[3], leaves[4], tab)
    leaves[0].grad = None
    a.sum().backward()  # k_out has no gradient: zeros
    ones = qr.norm_rope_bwd(to64(q), to64(wq), t64, np.ones(q.shape), 1e-6)
    assert np.all(np.abs(to64(leaves[0].grad) - ones[0]) <= 2.0 ** -8 * np.abs(ones[0]) + 2.0 ** -18 * ones[2])


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T,H,Hkv,D,bs,nb", [(1, 1, 1, 64, 16, 3), (5, 8, 2, 128, 16, 4), (133, 6, 6, 64, 32, 9),
                                             (700, 32, 8, 128, 256, 5)])
def test_append_against_oracle(T, H, Hkv, D, bs, nb, norm):
    q, k, v = I.randn_bf16((T, H, D), 60), I.randn_bf16((T, Hkv, D), 61), I.randn_bf16((T, Hkv, D), 62)
    wq, wk = (_weights(D, torch.float32, 63), _weights(D, torch.float32, 64)) if norm else (None, None)
    rng = np.random.default_rng(T)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    pos = rng.integers(0, 500, T).astype(np.int32)
    pad = rng.random(T) < 0.2 if T > 1 else np.zeros(1, bool)
    slots[pad], pos[pad] = -1, 10 ** 9  # a padding token's position is not looked at
    tab = s2().rope_table(500, D, 1.0)
    kc, vc = I.randn_bf16((nb, bs, Hkv, D), 65), I.randn_bf16((nb, bs, Hkv, D), 66)
    kd, vd = kc.cuda(), vc.cuda()
    q_out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = s2().cache_append(q.cuda(), k.cuda(), v.cuda(), tab, torch.from_numpy(pos).cuda(),
                            torch.from_numpy(slots).cuda(), kd, vd, w_q=None if wq is None else wq.cuda(),
                            w_k=None if wk is None else wk.cuda(), eps=EPS, q_out=q_out)
    torch.cuda.synchronize()
    assert s2().device_status() == 0
    live = ~pad
    t64 = to64(tab)[pos[live]]
    w64 = (None, None) if wq is None else (to64(wq), to64(wk))
    ref_q = qr.norm_rope(to64(q)[live], w64[0], t64, EPS)
    assert np.all(np.abs(to64(got)[live] - ref_q) <= _fwd_bound(to64(q)[live], w64[0], t64, ref_q))
    assert np.all(to64(got)[pad] == 7.0)
    ref_k = qr.norm_rope(to64(k)[live], w64[1], t64, EPS)
    gk, gv = to64(kd).reshape(nb * bs, Hkv, D), to64(vd).reshape(nb * bs, Hkv, D)
    assert np.all(np.abs(gk[slots[live]] - ref_k) <= _fwd_bound(to64(k)[live], w64[1], t64, ref_k))
    assert np.array_equal(gv[slots[live]], to64(v)[live])
    rest = np.setdiff1d(np.arange(nb * bs), slots[live])  # everything else as it was
    assert np.array_equal(gk[rest], to64(kc).reshape(nb * bs, Hkv, D)[rest])
    assert np.array_equal(gv[rest], to64(vc).reshape(nb * bs, Hkv, D)[rest])


def test_append_reports_positions_and_slots_out_of_range():
    T, H, D = 4, 2, 64
    q = I.randn_bf16((T, H, D), 70).cuda()
    tab = s2().rope_table(10, D, 1.0)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for pos, slots in (([0, 10, 2, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 16, 2, 3]), ([0, -1, 2, 3], [0, 1, 2, 3])):
        kc = torch.zeros(1, 16, H, D, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        s2().cache_append(q, q, q, tab, i32(pos), i32(slots), kc, kc.clone(), q_out=out)
        assert s2().device_status() == 7  # S2ATTN_ERR_DEVICE_BOUNDS
        assert s2().device_status() == 0  # read and cleared
        assert (out[1] == 0).all() and (kc[0, 1] == 0).all() and (out[0] != 0).any() and (kc[0, 3] != 0).any()


def test_other_stream_and_captured_graph():
    q, k, wq, wk, gq, gk = (t.cuda() for t in _case(1, 200, 4, 2, 128, torch.bfloat16, seed=80))
    tab = s2().rope_table(200, 128, 1.0)
    want = (*s2().qknorm_rope_forward(q, k, wq, wk, tab), *s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = (*s2().qknorm_rope_forward(q, k, wq, wk, tab), *s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab))
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    qs = q.clone()
    with torch.cuda.graph(g):
        cap = (*s2().qknorm_rope_forward(qs, k, wq, wk, tab), *s2().qknorm_rope_backward(qs, k, wq, wk, gq, gk, tab))
    for x in (q, k.repeat(1, 1, 2, 1), q):
        qs.copy_(x)
        g.replay()
        ref = (*s2().qknorm_rope_forward(x, k, wq, wk, tab), *s2().qknorm_rope_backward(x, k, wq, wk, gq, gk, tab))
        assert all(torch.equal(a, b) for a, b in zip(ref, cap))


def test_autograd_captured_with_its_gradients():
    B, N, H, Hkv, D, G = 1, 512, 4, 2, 64, 256
    q, k, wq, wk, do, _ = (t.cuda() for t in _case(B, N, H, Hkv, D, torch.float32, seed=90))
    v = I.randn_bf16((B, N, Hkv, D), 95).cuda()
    tab = s2().rope_table(N, D, 1.0)

    def step():
        leaves = [t.detach().requires_grad_() for t in (q, k, v, wq, wk)]
        o = s2().s2_qknorm_attn(*leaves, G, tab)
        return (o.detach(), *torch.autograd.grad(o, leaves, do))

    want = step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_python_refusals_on_the_gpu():
    q, k, wq, wk, gq, gk = (t.cuda() for t in _case(1, 32, 4, 2, 64, torch.float32))
    tab = s2().rope_table(32, 64, 1.0)
    f = s2().qknorm_rope_forward
    with pytest.raises(ValueError, match="contiguous"):
        f(q.transpose(1, 2).contiguous().transpose(1, 2), k, wq, wk, tab)
    with pytest.raises(ValueError, match="bfloat16"):
        f(q.float(), k, wq, wk, tab)
    with pytest.raises(ValueError, match="w_q"):
        f(q, k, wq.half(), wk, tab)
    with pytest.raises(ValueError, match="w_k"):
        f(q, k, wq, wk.bfloat16(), tab)
    with pytest.raises(ValueError, match="table"):
        f(q, k, wq, wk, tab[:16])
    with pytest.raises(ValueError, match="expected cuda"):
        s2().api._need("k", torch.zeros(1, device="cuda"), (1,), torch.float32, torch.device("cuda", 1))
    with pytest.raises(s2().S2AttnError, match="INVALID"):
        f(q, k, wq, wk, tab, eps=0.0)
    with pytest.raises(s2().S2AttnError, match="WORKSPACE"):
        s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab, workspace=torch.zeros(16, device="cuda"))
    with pytest.raises(ValueError, match="dq has shape"):
        s2().qknorm_rope_backward(q, k, wq, wk, gq, gk, tab, dq=gk)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        x = q.detach().requires_grad_()
        y, _ = s2().QKNormRope.apply(x, k, wq, wk, tab)
        g, = torch.autograd.grad(y, x, gq.detach().requires_grad_(), create_graph=True)
        g.sum().backward()
