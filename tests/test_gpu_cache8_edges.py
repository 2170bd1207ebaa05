"""The live 8-bit cache on the GPU at the borders of what it admits."""
import math

import pytest
import torch

import cache8_ref as R
from kv_cache_page_gb300 import cache8
from test_gpu_cache8 import _attend, _check

pytestmark = pytest.mark.gpu
DEV = "cuda"


class _Random:
    """A cache of random codes whose pages the sequences of any batch share (attention reads alone)."""

    def __init__(self, *, H, G, D, T, most_len, seed, dtype="bf16"):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.H, self.HQ, self.D, self.T, self.pages = H, H * G, D, T, 300
        self.width = -(-most_len // T)
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float16
        self.cache = cache8.Cache8(dtype=dtype, head_dim=D, num_kv_heads=H, num_q_heads=self.HQ, block_tokens=T,
                                   num_blocks=self.pages)
        codes = [torch.randint(0, 126, (self.pages, T, H, D), generator=self.g, dtype=torch.uint8, device=DEV)
                 for _ in range(2)]
        self.layer = cache8.Layer(*codes, *(torch.full((self.pages, H), 2.0 ** -7, device=DEV) for _ in range(2)))

    def batch(self, lens, new=None):
        n = len(lens)
        tables = torch.randint(0, self.pages, (n, self.width), generator=self.g, dtype=torch.int32, device=DEV)
        cu = None
        if new is not None:
            cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
        return cache8.Batch(tables, torch.tensor(lens, dtype=torch.int32, device=DEV), cu,
                            n_new=sum(new) if new is not None else n, max_new=max(new) if new is not None else 1,
                            max_len=max(lens))

    def attend(self, batch, workspace):
        q = torch.randn(batch.n_new, self.HQ, self.D, generator=torch.Generator(device=DEV).manual_seed(batch.n_new),
                        device=DEV).to(self.dtype)
        out, lse = torch.full_like(q, 9.0), torch.full((batch.n_new, self.HQ), 9.0, device=DEV)
        self.cache.attend(self.layer, batch, q, out, lse=lse, workspace=workspace)
        return out, lse


def test_one_workspace_for_batches_of_every_size():
    """Zero-filled once: sequences come and go, prompts join, and another cache uses it; every call gives what a
    workspace of its own gives."""
    a = _Random(H=8, G=4, D=64, T=16, most_len=8192, seed=1)
    b = _Random(H=2, G=7, D=128, T=16, most_len=8192, seed=2, dtype="fp16")
    c = _Random(H=1, G=4, D=256, T=5, most_len=1500, seed=3)
    steps = [(a, [8192 - 7 * s for s in range(n)], None) for n in (4, 8, 9, 64, 9, 33)]
    steps += [(a, [3000, 900, 8192, 5000, 77], [700, 1, 1, 20, 3]), steps[3]]
    steps += [(b, [8000, 5000], None), (b, [6000] * 40, None), (c, [1500, 700], [300, 4]), steps[1], steps[5],
              (b, [8192] * 12, [1, 5] * 6), steps[3]]
    calls = [(x, x.batch(lens, new)) for x, lens, new in steps]
    sizes = [x.cache.attend_workspace(batch) for x, batch in calls]
    assert min(sizes) > 0
    shared = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    for i, (x, batch) in enumerate(calls):
        own = torch.zeros(sizes[i], dtype=torch.uint8, device=DEV)
        want, got = x.attend(batch, own), x.attend(batch, shared)
        for w, g in zip(want, got):
            assert torch.equal(w, g), i
        assert not bool((want[0] == 9.0).all(-1).any()), i


def _fill_pages(su, k_of, v_of):
    """Every sequence's pages from values(n) times a factor of the page: k_of(i), v_of(i) for page i of a sequence."""
    for s, n in enumerate(su.lens):
        if n:
            fk, fv = (torch.tensor([f(t // su.T) for t in range(n)], dtype=torch.float64)[:, None, None]
                      for f in (k_of, v_of))
            k, v = (su.values(n).double() * f for f in (fk, fv))
            su.ref.write(su.tables[s], 0, (k.to(su.dtype), v.to(su.dtype)))


V_FACTORS = [[0.0, 1.0, 2.0 ** 70], [1.0, 0.0, 2.0 ** 100], [2.0 ** 119, 0.0, 0.0, 2.0 ** 80], [0.0, 2.0 ** 79], [0.0, 0.0, 2.0 ** 60]]


@pytest.mark.parametrize("T", [16, 24])
@pytest.mark.parametrize("factors", V_FACTORS)
@pytest.mark.parametrize("new", [None, [3, 9, 1], [80, 30, 64]])
def test_v_scales_far_apart(T, factors, new):
    """Zero pages (scale 2^-60) next to pages of very large values: the sum of the weights knows no scale of V."""
    lens = [90, 200, 64]
    su = R.Setup(D=64, H=1, T=T, lens=lens, dtype="bf16", seed=T)
    _fill_pages(su, lambda i: 0.25, lambda i: factors[i % len(factors)])
    for window in (0, 50):
        q, out, lse = _attend(su, lens, new, 32, window=window)
        _check(su, lens, new, q, out, lse, window=window)


@pytest.mark.parametrize("T", [16, 24])
@pytest.mark.parametrize("new", [None, [3, 9, 1], [80, 30, 64]])
@pytest.mark.parametrize("which", [2, 1])
def test_zero_keys_under_tiny_queries_are_keys(T, new, which):
    """Pages of zero keys (scale 2^-60) and query rows of 1e-30: the products of the factors leave FP32's range, the
    keys still count.  which: one page of `which` holds zeros."""
    lens = [90, 200, 64]
    su = R.Setup(D=64, H=1, T=T, lens=lens, dtype="bf16", seed=4)
    _fill_pages(su, lambda i: 0.0 if i % which == 0 else 1.0, lambda i: 1.0)
    q = su.queries(sum(new) if new else 3, 32).double()
    q[:, 8:24] *= 1e-30
    q = q.to(su.dtype)
    for window in (0, 50):
        _, out, lse = _attend(su, lens, new, 32, window=window, q=q)
        _check(su, lens, new, q, out, lse, window=window)


@pytest.mark.parametrize("T", [1, 5, 16, 24, 48])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [None, [3, 1, 9, 2], [70, 33, 40, 64]])
def test_pages_freed_behind_the_window(T, causal, new):
    """Table entries of pages that no query of the batch sees are not looked at: no error, the same outputs."""
    lens, window = [300, 121, 90, 177], 20
    su = R.Setup(D=64, H=1, T=T, lens=lens, dtype="fp16", seed=T)
    su.fill()
    for s, n in enumerate(lens):
        first = n - (new[s] if new else 1) - window + 1
        su.tables[s, :max(0, first) // T] = -1
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, out, lse = _attend(su, lens, new, 32, causal=causal, window=window, errors=errors)
    _check(su, lens, new, q, out, lse, causal=causal, window=window)
    assert errors.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("T,G", [(16, 4), (24, 4), (16, 32)])
@pytest.mark.parametrize("new", [None, [3, 9], [80, 64]])
def test_values_next_to_the_largest(T, G, new):
    """V of 2^124: outputs are as large, sums over the keys before they are normalised would be infinite."""
    lens = [150, 1400]
    su = R.Setup(D=64, H=1, T=T, lens=lens, dtype="bf16", seed=7, spread=0.0)
    _fill_pages(su, lambda i: 0.01, lambda i: 2.0 ** 124)
    for s, n in enumerate(lens):  # one sign, so that they add up
        for pid in su.tables[s, :-(-n // T)].tolist():
            su.ref.codes[1][pid] &= 0x7F
    q, out, lse = _attend(su, lens, new, G)
    _check(su, lens, new, q, out, lse)
    assert float(out.max()) > 2.0 ** 123


def test_arguments_that_do_not_fit_the_c_types():
    su = R.Setup(D=64, H=2, T=16, lens=[100], dtype="fp16")
    su.fill()
    for scale in (1e-60, 1e-300, 1e60):   # would become 0, which stands for 1 / sqrt(head_dim), or infinite
        with pytest.raises(ValueError):
            _attend(su, [100], None, 4, scale=scale)
    q, out, lse = _attend(su, [100], None, 4)
    for window in (2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 5):   # all of the sequence
        _, o, x = _attend(su, [100], None, 4, window=window, q=q)
        assert torch.equal(o, out) and torch.equal(x, lse), window
    assert math.isfinite(float(lse.max()))
