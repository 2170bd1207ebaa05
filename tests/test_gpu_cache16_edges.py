"""Attention over the live 16-bit cache where small faults would hide behind the outputs' own rounding."""
import math

import pytest
import torch

import cache16_ref as R
from cache16_cancel import PERIOD, SCALE, Cancel
from kv_cache_page_gb300 import cache8, cache16
from test_gpu_cache16 import _attend

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


# ---------------------------------------------------------------- what a row sees
@pytest.mark.parametrize("D,T", [(32, 16), (64, 5), (128, 16), (256, 24)])
@pytest.mark.parametrize("G,new", [(4, None), (2, [3, 6]), (8, [3, 6]), (16, [1, 4])])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_key_of_weight_0_is_seen_all_the_same(D, T, G, new, dtype, value):
    """A key whose score is -inf weighs nothing, and rows that see it are what they are without it; but 0 times a value that
    is no number is no number, whether or not the tile holds rows that do not see the key."""
    lens = [40, 64]
    su = R.Setup(D=D, H=1, T=T, lens=lens, dtype=dtype, seed=1)
    su.fill()
    n = sum(new) if new else 2
    q = su.values(n, G)
    q[..., 7] = q[..., 7].abs() + 0.5
    at = [lens[0] - (new[0] if new else 1), 62 if new else 50]  # (with several rows: some do not see it)
    for s, p in enumerate(at):
        pid = int(su.tables[s, p // T])
        su.pool[0][pid, p % T, 0, 7] = -math.inf
        su.pool[1][pid, p % T, 0, 3] = value
    pid = int(su.tables[1, 10 // T])
    su.pool[0][pid, 10 % T, 0, 7] = -math.inf  # one with a value that is a number
    q, out, lse = _attend(su, lens, new, G, q=q)
    tokens, gone = su.tokens, [[at[0]], [at[1], 10]]

    def without(role, s, m):
        x, ok = tokens(role, s, m)
        ok[[p for p in gone[s] if p < m]] = False
        return x, ok

    su.tokens = without
    row = 0
    for s, c in enumerate(new or [1, 1]):
        sees = torch.arange(lens[s] - c, lens[s]) >= at[s]
        o = out[row:row + c]
        assert torch.equal(torch.isfinite(o[..., 3]), ~sees[:, None].expand(c, G)), s
        o[..., 3] = torch.where(sees[:, None], 0.0, o[..., 3])
        want, wl, eo, el = su.attend(s, lens[s], q[row:row + c])
        want[..., 3] = torch.where(sees[:, None], 0.0, want[..., 3])
        assert bool(((o - want).abs() <= eo).all()) and bool(((lse[row:row + c] - wl).abs() <= el).all()), s
        row += c


@pytest.mark.parametrize("new", [None, [3, 2]])
def test_rows_whose_scores_are_all_minus_infinity(new):
    """They get what a row that sees no key gets."""
    lens = [5, 40]
    su = R.Setup(D=64, H=1, T=16, lens=lens, dtype="bf16", seed=1)
    su.fill()
    for s, n in enumerate(lens):
        for p in range(n):
            su.pool[0][int(su.tables[s, p // 16]), p % 16, 0, 7] = -math.inf
    n = sum(new) if new else 2
    q = su.values(n, 4)
    q[..., 7] = 1.0
    _, out, lse = _attend(su, lens, new, 4, q=q)
    assert not out.any() and bool((lse == -math.inf).all())
