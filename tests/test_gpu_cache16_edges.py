"""Attention over the live 16-bit cache where small faults would hide behind the outputs' own rounding."""
import math

import pytest
import torch

import cache16_ref as R
from cache16_cancel import PERIOD, SCALE, Cancel
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


# ---------------------------------------------------------------- every key once
def _counted(lens, new, *, D, H, T, G, dtype, layout="nhd", causal=True, window=0, seed=0):
    """All scores 0 and V 1 in one dim, another every 16 tokens: lse is the logarithm of the number of keys, and out how often
    each dim came up among them.  FP32 holds every sum exactly, so a lost or doubled step of any part shows."""
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, layout=layout, seed=seed)
    top = max(lens)
    for s, n in enumerate(lens):
        j = torch.arange(n)
        page, slot = su.tables[s].long()[j // T], j % T
        su.pool[0][page, slot] = 0.0
        for h in range(H):
            one = torch.zeros(n, D, dtype=su.dtype)
            one[j, (j // 16 + s + 3 * h) % D] = 1.0
            su.pool[1][page, slot, h] = one
    q, out, lse = _attend(su, lens, new, H * G, causal, window)
    before = torch.zeros(top + 1, D, dtype=torch.int32)  # [j]: how often each dim came up in tokens below j of sequence 0, head 0
    before[torch.arange(top) + 1, torch.arange(top) // 16 % D] = 1
    before = before.cumsum(0).double()
    half, least = torch.finfo(su.dtype).eps / 2, torch.finfo(su.dtype).tiny * torch.finfo(su.dtype).eps
    row = 0
    for s, c in enumerate(new if new is not None else [1] * len(lens)):
        n, at = lens[s], torch.arange(lens[s] - c, lens[s])
        hi = torch.where(at >= 0, at + 1 if causal else torch.full_like(at, n), 0)
        lo = torch.minimum((at - window + 1).clamp(min=0), hi) if window else torch.zeros_like(at)
        keys = (hi - lo).double()
        got = lse[row:row + c]
        want = torch.log(keys)[:, None].expand(c, H * G)
        # log2f within two units of its last place, one rounding after it
        assert torch.equal(torch.isneginf(got), torch.isneginf(want)), s
        f = torch.isfinite(want)
        assert bool(((got - want).abs()[f] <= want[f] * 2.0 ** -21 + 2.0 ** -22).all()), (s, float((got - want).abs()[f].max()))
        for h in range(H):
            o = out[row:row + c, h * G:h * G + G]
            x = ((before[hi] - before[lo]) / keys.clamp(min=1)[:, None]).roll((s + 3 * h) % D, 1)[:, None]
            # two FP32 roundings, one to the type
            assert bool(((o - x).abs() <= x * (half + 2.0 ** -22) + least).all()), (s, h, float((o - x).abs().max()))
        row += c


@pytest.mark.parametrize("D,T,H,G,dtype,layout", [(32, 16, 3, 1, "fp16", "nhd"), (64, 5, 1, 16, "bf16", "hnd"),
                                                  (128, 16, 2, 4, "bf16", "packed"), (256, 32, 1, 4, "fp16", "nhd")])
def test_every_key_once_in_equal_shares(D, T, H, G, dtype, layout):
    """More jobs than half the CTAs: shares that begin and end inside long jobs and go over many short ones."""
    lens = [20000, 3, 0, 1, 900, 0, 0, 4097] + [1 + (7 * i) % 90 for i in range(200)] + [0, 15000]
    for window in (0, 4000):
        _counted(lens, None, D=D, H=H, T=T, G=G, dtype=dtype, layout=layout, window=window)


@pytest.mark.parametrize("D,T,H,G,dtype", [(32, 16, 1, 8, "bf16"), (64, 24, 2, 2, "fp16"), (128, 16, 1, 20, "bf16"),
                                           (256, 5, 2, 4, "fp16")])
@pytest.mark.parametrize("lens", [[40001], [9000, 17, 0, 30000], [700, 20, 650, 81], [1000] * 36])
def test_every_key_once_in_even_parts(D, T, H, G, dtype, lens):
    _counted(lens, None, D=D, H=H, T=T, G=G, dtype=dtype)


@pytest.mark.parametrize("D,T,H,G,dtype", [(32, 16, 2, 4, "bf16"), (64, 24, 1, 5, "fp16"), (128, 16, 1, 2, "fp16"),
                                           (256, 16, 1, 16, "bf16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 333), (False, 0)])
def test_every_key_once_for_drafts(D, T, H, G, dtype, causal, window):
    lens, new = [9000, 5, 0, 3000, 777, 12], [4, 7, 2, 1, 40, 12]
    _counted(lens, new, D=D, H=H, T=T, G=G, dtype=dtype, causal=causal, window=window)


@pytest.mark.parametrize("D,T,H,G,dtype,layout", [(64, 16, 1, 8, "bf16", "packed"), (128, 16, 2, 4, "fp16", "nhd"),
                                                  (32, 5, 1, 3, "fp16", "hnd"), (256, 16, 1, 2, "bf16", "packed")])
@pytest.mark.parametrize("window", [0, 500])
def test_every_key_once_for_prompts(D, T, H, G, dtype, layout, window):
    """Prompts of thousands of tokens, one continued, next to a single token: thousands of tiles."""
    _counted([3001, 1, 2500, 1777], [3001, 1, 2500, 600], D=D, H=H, T=T, G=G, dtype=dtype, layout=layout, window=window)


@pytest.mark.parametrize("D,H,G,dtype", [(128, 2, 4, "bf16"), (64, 1, 7, "fp16")])
def test_prompts_of_real_length(D, H, G, dtype):
    """Values of every kind: rows at the ends of tiles and pages, and some between, against the definition."""
    lens, new = [2600, 40, 1900], [2600, 40, 700]
    su = R.Setup(D=D, H=H, T=16, lens=lens, dtype=dtype, seed=6, layout="packed")
    su.fill()
    q, out, lse = _attend(su, lens, new, H * G)
    row = 0
    for s, c in enumerate(new):
        start = lens[s] - c
        for i in sorted({0, 1, c - 1, c - 2} | {i for i in range(c) if (start + i) % 16 in (15, 0) and (start + i) % 400 < 32} |
                        set(range(7, c, 331))):
            want, wl, eo, el = su.attend(s, start + i + 1, q[row + i:row + i + 1])
            assert bool(((out[row + i] - want[0]).abs() <= eo[0]).all()) and bool(((lse[row + i] - wl[0]).abs() <= el[0]).all()), (s, i)
        row += c
