"""Attention over the live 16-bit cache on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import cache16_ref as R
from kv_cache_page_gb300 import cache8, cache16

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _attend(su, lens, new, HQ, causal=True, window=0, scale=None, hints=True, q=None, errors=None, layer=None, ws=None):
    c = su.cache(cache16, HQ)
    layer = layer or su.device_layer(cache16)
    n = sum(new) if new is not None else len(lens)
    q = su.values(n, HQ) if q is None else q
    b = su.batch(cache8, new, lens, errors=errors, hints=hints)
    ws = torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV) if ws is None else ws
    out = torch.full((n, HQ, su.D), 9.0, dtype=su.dtype, device=DEV)
    lse = torch.full((n, HQ), 9.0, device=DEV)
    c.attend(layer, b, q.to(DEV), out, lse=lse, causal=causal, window=window, scale=scale, workspace=ws)
    return q, out.cpu().double(), lse.cpu().double()


def _check(su, lens, new, q, out, lse, causal=True, window=0, scale=None):
    at = 0
    for s, n in enumerate(new if new is not None else [1] * len(lens)):
        if n == 0:
            continue
        want, wl, eo, el = su.attend(s, lens[s], q[at:at + n], causal, window, scale)
        o, x = out[at:at + n], lse[at:at + n]
        at += n
        assert torch.equal(torch.isneginf(x), torch.isneginf(wl)), s
        assert torch.equal(torch.isfinite(o), torch.isfinite(want)), s
        f = torch.isfinite(want)
        assert bool(((o - want).abs() <= eo)[f].all()), (s, float(((o - want).abs() / eo)[f].max()))
        g = torch.isfinite(wl)
        assert bool(((x - wl).abs() <= el)[g].all()), (s, float(((x - wl).abs() / el)[g].max()))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,G,layout,dtype", [(16, 2, 4, "nhd", "bf16"), (32, 1, 7, "hnd", "fp16"),
                                                (5, 3, 1, "packed", "fp16"), (1, 1, 16, "nhd", "bf16"),
                                                (48, 2, 20, "packed", "bf16"), (24, 1, 64, "hnd", "fp16")])
def test_step(D, T, H, G, layout, dtype):
    """One query a sequence: lengths 0, 1, around tiles and pages, jobs in one share and in several."""
    lens = [0, 1, 2, 15, 16, 17, 63, 129, 300, 1400]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, layout=layout, seed=D + G)
    su.fill()
    for hints in (True, False):
        q, out, lse = _attend(su, lens, None, H * G, hints=hints)
        _check(su, lens, None, q, out, lse)


@pytest.mark.parametrize("D,T,H,G,dtype", [(128, 16, 2, 4, "fp16"), (64, 24, 1, 5, "bf16"), (256, 16, 1, 2, "bf16"),
                                           (32, 5, 2, 1, "fp16"), (128, 1, 1, 8, "bf16"), (32, 64, 1, 20, "bf16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 13), (True, 64), (False, 0), (False, 40)])
def test_few_rows_masks(D, T, H, G, dtype, causal, window):
    """Drafted tokens and short chunks with every mask; idle sequences; more new tokens than held."""
    lens, new = [5, 40, 0, 130, 33, 2, 64], [5, 3, 2, 20, 0, 4, 1]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, seed=window)
    su.fill()
    q, out, lse = _attend(su, lens, new, H * G, causal, window)
    _check(su, lens, new, q, out, lse, causal, window)


@pytest.mark.parametrize("T,window", [(16, 0), (24, 0), (16, 1), (5, 50), (32, 130), (16, 2 ** 31 + 7)])
def test_windows_of_single_tokens(T, window):
    lens = [0, 1, 49, 50, 51, 200, 333, 128]
    su = R.Setup(D=64, H=2, T=T, lens=lens, dtype="bf16", layout="hnd", seed=T)
    su.fill()
    q, out, lse = _attend(su, lens, None, 8, window=window)
    _check(su, lens, None, q, out, lse, window=window)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 16), (256, 2)])
def test_whole_chunks(D, G):
    """Not what it is made for, but served: chunks of many rows next to single tokens."""
    lens, new = [100, 90, 1, 0, 77], [100, 33, 1, 0, 40]
    su = R.Setup(D=D, H=1, T=16, lens=lens, dtype="fp16", seed=5)
    su.fill()
    for causal, window in ((True, 0), (True, 20), (False, 0)):
        q, out, lse = _attend(su, lens, new, G, causal, window)
        _check(su, lens, new, q, out, lse, causal, window)


@pytest.mark.parametrize("new", [None, [4, 9, 1]])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_scores_of_every_size(new, dtype):
    """Scores that saturate the softmax, queries of tiny and large magnitude, a scale of the caller's."""
    lens = [90, 200, 64]
    su = R.Setup(D=64, H=2, T=16, lens=lens, dtype=dtype, seed=5, spread=1.5)
    su.fill()
    n = sum(new) if new else 3
    q = su.values(n, 8).double()
    q[:, 0] *= 1e-30
    q[:, 1] *= 30.0
    q[:, 2] *= 2.0 ** -7
    q[:, 3] = 0.0
    q = q.to(su.dtype)
    for scale in (None, 0.37):
        _, out, lse = _attend(su, lens, new, 8, q=q, scale=scale)
        _check(su, lens, new, q, out, lse, scale=scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("new", [None, [3, 9]])
def test_values_next_to_the_largest(dtype, new):
    """Outputs as large as V itself; sums over the keys before they are normalised would leave a smaller range."""
    lens = [150, 1400]
    su = R.Setup(D=64, H=1, T=16, lens=lens, dtype=dtype, seed=7, spread=0.0)
    big = torch.finfo(su.dtype).max
    for s, n in enumerate(lens):
        v = big * torch.rand(n, 1, 64, generator=su.g).clamp(min=0.5)
        su.put(s, 0, (0.01 * su.values(n).float()).to(su.dtype), v.clamp(max=0.99 * big).to(su.dtype))
    q, out, lse = _attend(su, lens, new, 4)
    _check(su, lens, new, q, out, lse)
    assert float(out.max()) > 0.6 * big


def test_weights_far_below_the_largest_still_count():
    """One key ahead of many by a factor that a single 16-bit weight would round away."""
    lens = [1200]
    for dtype in ("fp16", "bf16"):
        su = R.Setup(D=32, H=1, T=16, lens=lens, dtype=dtype, seed=2)
        k, v = torch.zeros(1200, 1, 32, dtype=su.dtype), torch.ones(1200, 1, 32, dtype=su.dtype)
        k[700, 0, 0] = 1.0
        v[700] = -1.0
        su.put(0, 0, k, v)
        q = torch.zeros(1, 4, 32, dtype=su.dtype)
        q[0, :, 0] = torch.tensor([20.0, 30.0, 45.0, 60.0])
        _, out, lse = _attend(su, lens, None, 4, q=q)
        _check(su, lens, None, q, out, lse)


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G,new", [(2, [3, 6]), (8, [3, 6]), (4, [1, 16])])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_arrive(D, G, new, value):
    """A key or value that is no number, of a later token, or of one behind the window, leaves other rows as they are."""
    lens = [40, 64]
    su = R.Setup(D=D, H=1, T=16, lens=lens, dtype="fp16", seed=1)
    su.fill()
    su.pool[1][int(su.tables[0, 2]), 39 - 32, 0, 5] = value           # value of sequence 0's last token
    su.pool[1][int(su.tables[1, 0]), 3, 0, 2] = value                 # behind a window of 20
    su.pool[0][int(su.tables[1, 0]), 4, 0, 2] = math.nan
    su.pool[0][int(su.tables[1, 3]), 62 - 48, 0, 9] = math.nan        # key of sequence 1's last but one token
    q, out, lse = _attend(su, lens, new, G, window=20)
    _check(su, lens, new, q, out, lse, window=20)
    assert not torch.isfinite(out).all() and torch.isfinite(out).any()


def test_a_query_that_is_no_number_stays_in_its_row():
    su = R.Setup(D=128, H=1, T=16, lens=[50], dtype="bf16")
    su.fill()
    q = su.values(1, 4)
    q[0, 1, 7] = math.nan
    q[0, 2, 8] = math.inf
    q, out, _ = _attend(su, [50], None, 4, q=q)
    bad = torch.isnan(out).any(-1)[0].tolist()
    assert bad[1] and not bad[0] and not bad[3]


@pytest.mark.parametrize("T", [16, 24])
@pytest.mark.parametrize("new", [None, [2, 1, 3, 2], [40, 40, 40, 40]])
def test_bad_pages(T, new):
    """Table entries that are no page, and lengths past the table: reported, skipped."""
    lens = [60, 60, 60, 300]
    su = R.Setup(D=64, H=2, T=T, lens=[60, 60, 60, 60], dtype="fp16", seed=2)
    su.fill()
    su.tables[1, 1] = su.pages
    su.tables[2, 0] = -5
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, out, lse = _attend(su, lens, new, 4, errors=errors)
    _check(su, lens, new, q, out, lse)
    assert errors.tolist() == [0, 1, 1, 1]


@pytest.mark.parametrize("T", [1, 5, 16, 24, 48])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [None, [3, 1, 9, 2]])
def test_pages_freed_behind_the_window(T, causal, new):
    """Table entries of pages that no query of the batch sees are not looked at: no error, the same outputs."""
    lens, window = [300, 121, 90, 177], 20
    su = R.Setup(D=64, H=1, T=T, lens=lens, dtype="fp16", seed=T)
    su.fill()
    for s, n in enumerate(lens):
        first = n - (new[s] if new else 1) - window + 1
        su.tables[s, :max(0, first) // T] = -1
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, out, lse = _attend(su, lens, new, 16, causal=causal, window=window, errors=errors)
    _check(su, lens, new, q, out, lse, causal=causal, window=window)
    assert errors.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("D,T,H,G", [(128, 16, 2, 4), (64, 16, 1, 16), (256, 32, 1, 4), (32, 16, 3, 1)])
def test_long_ones_next_to_many_short_ones(D, T, H, G):
    """Jobs over many shares, shares of many jobs, empty slots between them."""
    lens = [20000, 3, 0, 1, 900, 0, 0, 4097] + [1 + (7 * i) % 90 for i in range(200)] + [0, 15000]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype="bf16", seed=3)
    su.fill()
    q, out, lse = _attend(su, lens, None, H * G)
    _check(su, lens, None, q, out, lse)


def test_more_sequences_than_a_block_s_threads():
    lens = [(5 * i) % 37 for i in range(1500)]
    su = R.Setup(D=32, H=1, T=16, lens=lens, dtype="fp16", seed=3)
    su.fill()
    q, out, lse = _attend(su, lens, None, 2)
    _check(su, lens, None, q, out, lse)
    new = [(3 * i) % 4 for i in range(1500)]
    q, out, lse = _attend(su, lens, new, 2)
    _check(su, lens, new, q, out, lse)


def test_rows_past_the_caller_s_count_are_not_touched():
    """cu_new that promises more rows than n_new: the surplus is not read or written."""
    su = R.Setup(D=32, H=1, T=16, lens=[32, 32], dtype="fp16")
    su.fill()
    c, layer = su.cache(cache16, 1), su.device_layer(cache16)
    b = cache8.Batch(su.tables.to(DEV), torch.tensor([32, 32], dtype=torch.int32, device=DEV),
                     torch.tensor([0, 4, 900], dtype=torch.int32, device=DEV), n_new=10, max_new=6, max_len=32)
    mem = torch.full((64, 1, 32), 3.0, dtype=su.dtype, device=DEV)
    q = su.values(10).to(DEV)
    c.attend(layer, b, q, mem[:10], workspace=torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV))
    assert bool((mem[10:] == 3.0).all()) and not bool((mem[:10] == 3.0).all(-1).any())


@pytest.mark.parametrize("new", [None, [3, 1, 5]])
def test_same_result_every_time_and_on_another_stream(new):
    lens = [5000, 300, 1200]
    su = R.Setup(D=128, H=2, T=16, lens=lens, dtype="bf16")
    su.fill()
    c, layer = su.cache(cache16, 8), su.device_layer(cache16)
    n = sum(new) if new else 3
    q = su.values(n, 8).to(DEV)
    b = su.batch(cache8, new, lens)
    ws = torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV)
    outs, side = [], torch.cuda.Stream()
    for i in range(6):
        out, lse = torch.empty(n, 8, 128, dtype=su.dtype, device=DEV), torch.empty(n, 8, device=DEV)
        torch.cuda.synchronize()
        c.attend(layer, b, q, out, lse=lse, workspace=ws, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_one_workspace_for_every_batch_and_for_the_8_bit_cache():
    """Zero-filled once, used by batches of every size and by both caches in turn: each gives what a fresh one gives."""
    lens = [4000, 700, 64, 1, 0, 2500]
    su = R.Setup(D=64, H=2, T=16, lens=lens, dtype="fp16", seed=8)
    su.fill()
    c16, layer = su.cache(cache16, 8), su.device_layer(cache16)
    c8 = cache8.Cache8(dtype="fp16", head_dim=64, num_kv_heads=2, num_q_heads=8, block_tokens=16, num_blocks=su.pages)
    codes = [torch.randint(0, 126, (su.pages, 16, 2, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    layer8 = cache8.Layer(*codes, *(torch.full((su.pages, 2), 2.0 ** -7, device=DEV) for _ in range(2)))
    batches = [(su.batch(cache8, new, lens), n) for new, n in ((None, 6), ([3, 1, 2, 1, 0, 9], 16), ([1, 1, 1, 1, 1, 40], 45))]
    shared = torch.zeros(max(max(c16.attend_workspace(b), c8.attend_workspace(b)) for b, _ in batches), dtype=torch.uint8, device=DEV)
    for turn in range(2):
        for b, n in batches:
            q = su.values(n, 8).to(DEV)
            for c, y in ((c16, layer), (c8, layer8)):
                got = []
                for ws in (torch.zeros_like(shared), shared):
                    out, lse = torch.empty_like(q), torch.empty(n, 8, device=DEV)
                    c.attend(y, b, q, out, lse=lse, workspace=ws)
                    got.append((out, lse))
                assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("new", [None, [9, 1, 4]])
def test_hints_that_are_too_small_cost_time_alone(new):
    """max_new and max_len below what the arrays hold: every row is served all the same."""
    lens = [2100, 40, 700]
    su = R.Setup(D=64, H=1, T=16, lens=lens, dtype="bf16", seed=4)
    su.fill()
    n = sum(new) if new else 3
    c, layer, full = su.cache(cache16, 4), su.device_layer(cache16), su.batch(cache8, new)
    b = cache8.Batch(full.tables, full.lens, full.cu_new, n_new=n, max_new=1, max_len=1)
    q = su.values(n, 4)
    out, lse = torch.empty(n, 4, 64, dtype=su.dtype, device=DEV), torch.empty(n, 4, device=DEV)
    c.attend(layer, b, q.to(DEV), out, lse=lse, workspace=torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV))
    _check(su, lens, new, q, out.cpu().double(), lse.cpu().double())


def test_pages_shared_between_sequences():
    """A common prefix of whole pages in several tables."""
    lens = [100, 100, 70, 64]
    su = R.Setup(D=128, H=1, T=16, lens=lens, dtype="fp16", seed=4)
    su.fill()
    su.tables[1:, :4] = su.tables[0, :4]
    q, out, lse = _attend(su, lens, None, 8)
    _check(su, lens, None, q, out, lse)


@pytest.mark.parametrize("window", [0, 33, 90])
def test_tables_that_end_before_the_window(window):
    """Lengths past the table: what lies in it is seen where the window reaches it, and rows may see nothing at all."""
    lens = [200, 90, 50]
    su = R.Setup(D=64, H=2, T=16, lens=[48, 48, 48], dtype="bf16", seed=3)
    su.fill()
    errors = torch.zeros(3, dtype=torch.int32, device=DEV)
    q, out, lse = _attend(su, lens, None, 4, window=window, errors=errors)
    _check(su, lens, None, q, out, lse, window=window)
    assert errors.tolist() == [1, 1, 1]


def test_strided_queries_and_outputs():
    lens = [90, 17]
    su = R.Setup(D=64, H=2, T=16, lens=lens, dtype="bf16", seed=4)
    su.fill()
    c, layer, b = su.cache(cache16, 4), su.device_layer(cache16), su.batch(cache8)
    q = su.values(2, 4)
    wide = torch.full((2, 4, 3, 64), 5.0, dtype=su.dtype, device=DEV)
    wide[:, :, 0] = q.to(DEV)
    c.attend(layer, b, wide[:, :, 0], wide[:, :, 2], workspace=torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV))
    assert bool((wide[:, :, 1] == 5.0).all()) and torch.equal(wide[:, :, 0].cpu(), q)
    _, out, _ = _attend(su, lens, None, 4, q=q, layer=layer)
    assert torch.equal(wide[:, :, 2].cpu().double(), out)


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of K."""
    H, T, D = 8, 64, 256
    pages = (1 << 32) // (H * T * D * 2) + 20
    su = R.Setup(D=D, H=H, T=T, lens=[100], dtype="fp16")
    c = cache16.Cache16(dtype="fp16", head_dim=D, num_kv_heads=H, num_q_heads=2 * H, block_tokens=T, num_blocks=pages)
    layer = c.new_layer()
    high = [pages - 1, pages - 9]
    su.fill()
    for role, mem in enumerate((layer.k, layer.v)):
        for i, pid in enumerate(high):
            mem.view(pages, T, H, D)[pid] = su.pool[role][int(su.tables[0, i])].to(DEV)
    lens = torch.tensor([100], dtype=torch.int32, device=DEV)
    b = cache8.Batch(torch.tensor([high], dtype=torch.int32, device=DEV), lens, max_len=100)
    q = su.values(1, 2 * H)
    out, lse = torch.empty(1, 2 * H, D, dtype=su.dtype, device=DEV), torch.empty(1, 2 * H, device=DEV)
    c.attend(layer, b, q.to(DEV), out, lse=lse, workspace=torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV))
    _check(su, [100], None, q, out.cpu().double(), lse.cpu().double())


def test_refusals():
    su = R.Setup(D=64, H=2, T=16, lens=[600], dtype="fp16")
    c, layer, b = su.cache(cache16, 4), su.device_layer(cache16), su.batch(cache8)
    q = su.values(1, 4).to(DEV)
    out = torch.empty_like(q)
    ws = torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV)

    def code(f):
        with pytest.raises(cache16.KvCodecError) as e:
            f()
        return e.value.code

    assert code(lambda: c.attend(layer, b, q, out)) == -1                          # workspace missing
    assert code(lambda: c.attend(layer, b, q, out, workspace=ws[:-16])) == -1      # too small
    odd = torch.zeros(ws.numel() + 16, dtype=torch.uint8, device=DEV)[4:]
    assert code(lambda: c.attend(layer, b, q, out, workspace=odd)) == -5
    narrow = torch.zeros(1, 4 * 64, dtype=su.dtype, device=DEV)
    assert code(lambda: c.attend(layer, b, q, narrow.as_strided((1, 4, 64), (256, 32, 1)), workspace=ws)) == -3
    for f in (lambda: c.attend(layer, b, q[:, :2], out, workspace=ws), lambda: c.attend(layer, b, q.float(), out, workspace=ws),
              lambda: c.attend(layer, b, q, out, lse=torch.empty(1, 3, device=DEV), workspace=ws),
              lambda: c.attend(layer, b, q, out, scale=-1.0, workspace=ws), lambda: c.attend(layer, b, q, out, scale=1e-60, workspace=ws),
              lambda: c.attend(layer, b, q, out, window=-1, workspace=ws),
              lambda: c.attend(cache16.Layer(layer.k[1:], layer.v), b, q, out, workspace=ws),
              lambda: c.attend(cache16.Layer(layer.k.bfloat16(), layer.v.bfloat16()), b, q, out, workspace=ws),
              lambda: cache16.Layer(layer.k, layer.v.bfloat16()), lambda: cache16.Layer(layer.k.cpu(), layer.v)):
        with pytest.raises(ValueError):
            f()
    # no rows: nothing is launched
    empty = cache8.Batch(torch.zeros(0, 4, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    none = torch.empty(0, 4, 64, dtype=su.dtype, device=DEV)
    c.attend(layer, empty, none, none)
    assert c.attend_workspace(empty) == 0
