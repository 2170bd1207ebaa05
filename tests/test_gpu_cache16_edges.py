"""Attention over the live 16-bit cache where small faults would hide behind the outputs' own rounding."""
import math

import pytest
import torch

import cache16_ref as R
from cache16_cancel import PERIOD, SCALE, Cancel
from kv_cache_page_gb300 import cache8, cache16
from test_gpu_cache16 import _attend, _check

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- the weights of V
def _cancelling(D, dtype, n, T=16):
    su = R.Setup(D=D, H=1, T=T, lens=[n], dtype=dtype)
    c = Cancel(su.dtype)
    k, v, sign = c.tokens(n, D)
    su.put(0, 0, k, v)
    return su, c, sign


def _near(out, c, sign, dims=slice(None)):
    off = (out - c.out * sign).abs()[..., dims] / sign.abs()[dims]
    assert float(off.max()) <= c.bound(), float(off.max()) / c.bound()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,T,G", [(32, 16, 4), (64, 5, 16), (128, 16, 8), (256, 48, 1)])
def test_weights_are_as_fine_as_the_sums(D, T, G, dtype):
    """Single tokens over values that cancel: what is left would be another by far with weights of too few bits."""
    su, c, sign = _cancelling(D, dtype, 1600, T)
    q = torch.zeros(1, G, D, dtype=su.dtype)
    q[..., 0] = 1.0
    _, out, lse = _attend(su, [1600], None, G, q=q, scale=SCALE)
    _near(out, c, sign)
    # FP32 sums of 1600 weights, each and the logarithm within 2^-20
    assert float((lse - math.log(100 * c.sum)).abs().max()) < 1600 * 2.0 ** -24 + 2.0 ** -19


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,G", [(32, 1), (64, 1), (128, 2), (256, 1)])
@pytest.mark.parametrize("odd", [False, True])
def test_weights_of_chunks_are_as_fine_as_the_sums(D, G, dtype, odd):
    """Rows that see different keys; odd: with a value among them that only the last row sees and that is no number."""
    n = 160
    su, c, sign = _cancelling(D, dtype, n)
    if odd:
        su.pool[1][int(su.tables[0, -1]), 15, 0, 5] = math.nan
    q = torch.zeros(n, G, D, dtype=su.dtype)
    q[..., 0] = 1.0
    _, out, _ = _attend(su, [n], [n], G, q=q, scale=SCALE)
    ends = list(range(PERIOD - 1, n, PERIOD))
    _near(out[ends[:-1]], c, sign)
    _near(out[ends[-1]], c, sign, [d for d in range(D) if d != 5 or not odd])
    assert bool(torch.isnan(out[-1, :, 5]).all()) == odd
