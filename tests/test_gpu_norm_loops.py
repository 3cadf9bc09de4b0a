"""The norm's forward and backward and the append at sizes beyond one pass of
their grids (16 blocks of 256 threads an SM: 606,208 threads of work on 148
SMs), held to the bounds of the smaller shapes' tests.  In the backward a thread
then adds up at most 2 heads x 8 passes = 16 rows in sequence, where those bounds
allow 48."""
import pytest
import torch

from tests import test_gpu_qknorm as tq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,H,Hkv,D,wt", [(30011, 8, 2, 128, torch.bfloat16), (30011, 13, 5, 64, torch.float32)])
def test_norm_beyond_one_pass(N, H, Hkv, D, wt):
    lanes = N * (-(-H // 4) + -(-Hkv // 4)) * (D // 16)
    assert lanes > 148 * 16 * 256
    tq.test_forward_and_backward_against_oracle(1, N, H, Hkv, D, wt)


@pytest.mark.parametrize("norm", [True, False])
def test_append_beyond_one_pass(norm):
    T, H, Hkv, D = 20011, 8, 2, 128
    assert T * (2 + 2 * 1) * (D // 16) > 148 * 16 * 256
    tq.test_append_against_oracle(T, H, Hkv, D, 64, 320, norm)
