"""Rows take in the weights that they pick, and no others."""
import pytest
import torch

from mxfp4_block_scaled_02_amd import ops
from tests.test_gpu_moe import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 6, 3), (5, 256, 160, 6, 2), (5, 4128, 128, 12, 2), (10, 288, 96, 7, 1), (7, 256, 160, 6, 2), (16, 4128, 128, 9, 3), (16, 256, 128, 9, 4),
                                       (17, 256, 128, 9, 2), (20, 288, 96, 30, 5), (90, 288, 96, 4, 2), (500, 1024, 96, 8, 1)])
def test_an_expert_that_is_not_finite_changes_no_token_without_it(T, H, I, E, k, byte):
    """Both ways of the down product, and gate and up, hold tokens of several experts side by side."""
    x, ids, weights, (q13, s13), (q2, s2) = layer(T + H + byte, T, H, I, E, k)
    bad = int(ids[0, 0])
    hit = (ids == bad).any(dim=1)
    good = [ops.pack_experts(q13, s13), ops.pack_experts(q2, s2)]
    want = ops.moe_a16w4(x, ids, weights, *good, I)
    for which, (q, s) in enumerate([(q13, s13), (q2, s2)]):
        s = s.clone()
        s[bad] = byte
        packed = list(good)
        packed[which] = ops.pack_experts(q, s)
        y = ops.moe_a16w4(x, ids, weights, *packed, I)
        assert torch.equal(y[~hit], want[~hit])
        if byte == 255:
            assert not torch.isfinite(y[hit]).all(dim=1).any()
    assert torch.isfinite(want).all() and (T == 1 or bool((~hit).any()))
