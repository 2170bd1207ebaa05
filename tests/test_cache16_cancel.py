"""The cancelling keys and values of the GPU's test of the weights: that they tell the weights' roundings apart (no GPU)."""
import pytest
import torch

from cache16_cancel import PERIOD, Cancel, weight


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_coarser_weights_would_be_seen(dtype):
    """One 16-bit term of the weights is off by far more than the test's bound, two of BF16 by twice the bound at least;
    two of FP16 and three of BF16 are within it."""
    c = Cancel(dtype)
    assert c.off_with(1) > 100 * c.bound()
    if dtype is torch.bfloat16:
        assert c.off_with(2) > 2 * c.bound()
        assert c.off_with(3) < 0.05 * c.bound()
    else:
        assert c.off_with(2) < 0.5 * c.bound()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_what_is_left_is_small(dtype):
    c = Cancel(dtype)
    k, v, sign = c.tokens(3 * PERIOD, 32)
    assert torch.equal(k.double()[:PERIOD, 0, 0], c.keys) and torch.equal(v.double()[PERIOD:2 * PERIOD, 0], c.values[:, None] * sign)
    w = weight(k[:, 0, 0].double())
    out = (w[:, None] * v[:, 0].double()).sum(0) / w.sum()
    assert float((out - c.out * sign).abs().max()) < 1e-12 and abs(c.out) < 2.0 ** -13 * c.size and c.z < 2
