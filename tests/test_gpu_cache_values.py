"""Values of V that a product of the matrix units must not decide: infinite and
NaN values under weights that underflow.  exp of any finite score is more than
0, so a row that sees such a value is not finite, whatever the weight."""
import numpy as np
import pytest

from tests.test_gpu_cache import _batch, _call, kernel  # noqa: F401
from tests.parity_util import to64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (8, 2, 128), (16, 1, 128)])
@pytest.mark.parametrize("lens", [[(0, 3)], [(40, 6), (125, 5), (1000, 2), (62, 4)]])
def test_non_finite_value_under_a_vanishing_weight(kernel, lens, H, Hkv, D, tree):  # noqa: F811
    """Draft 1 scores 256 less than draft 0 (exp(-256) is 0 in 32 bits); its V has inf and NaN."""
    masks = None
    if tree:  # every draft sees itself, draft 0 and, where odd, draft 1
        masks = [np.array([1 << j | 1 | (2 if j & 1 else 0) for j in range(n)], np.uint64) for _, n in lens]
    b = _batch(lens, H, Hkv, D, 16, masks, 31)
    b["q"].fill_(4.0)
    top = 128.0 / (4 * D / np.sqrt(D))   # a key of this height scores 128
    for r, (c, n) in enumerate(lens):
        k, v = b["reqs"][r]
        k.zero_()
        k[c], k[c + 1] = top, -top
        v[c + 1, :, 3], v[c + 1, :, D - 1] = float("inf"), float("nan")
        p = np.arange(c + n)
        b["kc"][b["tab"][r, p // 16], p % 16], b["vc"][b["tab"][r, p // 16], p % 16] = k, v
    o, _ = _call(b)
    o = to64(o)
    for r, (c, n) in enumerate(lens):
        for j in range(n):
            sees = j >= 1 if masks is None else bool(int(masks[r][j]) & 2)
            row = o[b["cu"][r] + j]
            assert np.isfinite(row[:, 4:D - 1]).all() and np.isfinite(row[:, :3]).all(), (r, j)
            assert np.isfinite(row[:, [3, D - 1]]).all() == (not sees) and (not sees or not np.isfinite(row[:, [3, D - 1]]).any()), (r, j)
