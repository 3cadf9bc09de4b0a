"""Which form of the few-row kernel a single request takes at lengths beyond the
clusters' limit: clusters only where they were measured faster (they fill the
resident CTAs), equal runs and a join elsewhere.  Results do not depend on it."""
import pytest
import torch

import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import _lib, inputs as I

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,D,launches", [
    (24, 128, 1), (32, 128, 1), (36, 128, 2), (48, 128, 1), (64, 128, 1), (96, 128, 2), (112, 128, 1), (128, 128, 1),
    (192, 128, 2), (224, 128, 1), (256, 128, 1), (257, 128, 2),
    (24, 64, 2), (28, 64, 2), (32, 64, 1), (48, 64, 2), (64, 64, 1), (96, 64, 2), (128, 64, 2), (256, 64, 2),
])
def test_form_of_a_long_request(heads, D, launches):
    kc, vc = (I.randn_bf16((4, 64, heads, D), i).cuda() for i in (1, 2))
    q = I.randn_bf16((1, heads, D), 3).cuda()
    tab = torch.full((1, 1000), -1, dtype=torch.int32, device="cuda")   # room for 64000 keys
    tab[0, :4] = torch.arange(4)
    ctx, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([200], [0, 1]))
    o, lse = s2.cache_attention(q, kc, vc, tab, ctx, cu)
    assert _lib.s2attn_last_launch_count() == launches
    _lib.s2attn_set_tile_override("cache=" + ("dec" if launches == 1 else "cluster"))
    try:
        o2, lse2 = s2.cache_attention(q, kc, vc, tab, ctx, cu)
    finally:
        _lib.s2attn_set_tile_override(None)
    # the forms split the keys differently: o rounded to bf16 once more or less (2^-8), weights 2^-8 of the mean of |v| < 5
    assert ((o.float() - o2.float()).abs() <= 2 ** -7 * o.abs().float() + 2 * 2 ** -8 * 5).all()
    assert ((lse - lse2).abs() <= 2 ** -13).all() and s2.device_status() == 0
