"""The short compiled way into the norm and decoding calls (csrc/s2_torch.cpp)
against the Python one: it takes the usual case only, with the same bits, and
leaves everything else -- wrong operands above all -- to the Python checks."""
import pytest
import torch

import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import _lib, api

NAMES = ("qknorm_fwd", "qknorm_bwd", "cache_append", "cache_plan", "cache_attention")


@pytest.fixture
def fast():
    """The bound functions; skipped where the extension is not built for this torch."""
    pytest.importorskip("sparse_attention_attn_b200._s2torch")
    return {n: getattr(api._fast, n) for n in NAMES}


def _args(dev, T=5, H=4, Hkv=2, D=64, bs=16):
    """Operands of every call: one set of tensors of two requests."""
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16().to(dev)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    w_q, w_k = (torch.rand(D, generator=g).to(dev) + 0.5 for _ in range(2))
    table = torch.randn(64, D // 2, 2, generator=g).to(dev)
    q, k = bf(1, T, H, D), bf(1, T, Hkv, D)
    kc, vc = bf(6, bs, Hkv, D), bf(6, bs, Hkv, D)
    tab = i32(4, 1, 0, -1, 2, -1).reshape(2, 3)
    return {
        "qknorm_fwd": [q, k, w_q, w_k, table[:T], 1e-6],
        "qknorm_bwd": [q, k, w_q, w_k, bf(1, T, H, D), bf(1, T, Hkv, D), table[:T], 1e-6],
        "cache_append": [q[0], k[0], bf(T, Hkv, D), table, i32(*range(7, 7 + T)), i32(*range(3, 3 + T)), kc, vc, w_q, w_k,
                         1e-6, None],
        "cache_plan": [i32(30, 9), i32(3, 2), tab, i32(5, 3), bs, T, i32(-1, 0, 0, -1, 0)],
        "cache_attention": [q[0], kc, vc, i32(4, 1, 0, 5, 2, 3).reshape(2, 3), i32(30, 9), i32(0, 3, 5),
                            torch.tensor([1, 3, 5, 1, 3], device=dev)],
    }


def test_cpu_tensors_and_other_objects_are_left_to_python(fast):
    for name, args in _args("cpu").items():
        assert fast[name](*args) is None, name
        assert fast[name](*args[:-1]) is None and fast[name]() is None
        for bad in (None, 3, "x", [1.0], object()):
            assert fast[name](*([bad] * len(args))) is None
    from sparse_attention_attn_b200 import _s2torch
    with pytest.raises(TypeError):
        _s2torch.bind(1, 2)
    with pytest.raises((TypeError, ValueError)):
        _s2torch.bind(*([0] * 7))


class _Without:
    def __getattr__(self, name):
        return lambda *args: None


def _copies(a):
    return [x.clone() if isinstance(x, torch.Tensor) else x for x in a]


def _public(name, a):
    """The public call with these operands: every tensor it returns or writes."""
    if name == "qknorm_fwd":
        return s2.qknorm_rope_forward(*a)
    if name == "qknorm_bwd":
        return s2.qknorm_rope_backward(*a)
    if name == "cache_append":
        return [s2.cache_append(*a), a[6], a[7]]
    if name == "cache_plan":
        return [*s2.cache_plan(*a), a[2]]
    return s2.cache_attention(*a)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_same_bits_both_ways(fast, monkeypatch, name):
    args = _args("cuda")[name]
    assert fast[name](*_copies(args)) is not None
    got = _public(name, _copies(args))
    monkeypatch.setattr(api, "_fast", _Without())
    want = _public(name, _copies(args))
    torch.cuda.synchronize()
    assert s2.device_status() == 0
    for x, y in zip(got, want, strict=True):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_wrong_operands_are_refused_by_name(fast, name):
    """Each tensor in turn of another type, device or shape, or with a stride."""
    good = _args("cuda")[name]
    for i, t in enumerate(good):
        if not isinstance(t, torch.Tensor):
            continue
        wide = torch.empty((*t.shape, 2), dtype=t.dtype, device="cuda")[..., 0]
        for bad in (t.to(torch.float16), t.cpu(), t[None], wide, t.cpu().numpy() if t.dtype != torch.bfloat16 else 1):
            a = [*good]
            a[i] = bad
            assert fast[name](*a) is None, (i, str(bad)[:200])
            with pytest.raises((ValueError, TypeError, AttributeError, _lib.S2AttnError)):
                _public(name, a)
