"""The live 8-bit cache on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import cache8_ref as R
from kv_cache_page_gb300 import cache8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _write_case(su, lens, new, HQ=None, kv=None):
    """The new tokens of `new` (the last of lens) written on the device and by the reference; both caches."""
    c = su.cache(cache8, HQ or su.H)
    layer = su.device_layer(cache8)
    rows = sum(new)
    k, v = kv if kv is not None else (su.values(rows), su.values(rows))
    c.write(layer, su.batch(cache8, new, lens), k.to(DEV), v.to(DEV))
    at = 0
    for s, n in enumerate(new):
        su.ref.write(su.tables[s], lens[s] - n, (k[at:at + n], v[at:at + n]))
        at += n
    return c, layer


def _same(su, layer):
    for role, codes in enumerate(su.codes_of(layer)):
        assert torch.equal(codes, su.ref.codes[role]), role
        got = (layer.k_scale, layer.v_scale)[role].cpu().double()
        assert torch.equal(torch.nan_to_num(got, nan=-1), torch.nan_to_num(su.ref.scale[role], nan=-1)), role


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,by_head,dtype", [(16, 8, False, "bf16"), (32, 2, True, "fp16"), (5, 3, False, "fp16"),
                                               (1, 1, True, "bf16"), (130, 1, False, "bf16")])
def test_write(D, T, H, by_head, dtype):
    """Bit for bit: fresh pages, half-filled pages whose scale stays or grows, one token, none."""
    new = [1, 0, 3, 40, 17, 1, 2 * T, 1]
    lens = [1, 7, 3, 61, 33, T + 1, 2 * T, 2 * T]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, by_head=by_head, seed=D + T)
    su.fill([n - c for n, c in zip(lens, new)])
    _, layer = _write_case(su, lens, new)
    _same(su, layer)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_one_token_at_a_time_equals_the_reference(dtype):
    su = R.Setup(D=64, H=2, T=16, lens=[20, 37], dtype=dtype, spread=2.0)
    c, layer = su.cache(cache8, 2), su.device_layer(cache8)
    for step in range(37):
        lens = [min(step + 1, 20), step + 1]
        k, v = su.values(2), su.values(2)
        live = [1 if step < 20 else 0, 1]
        new = [i for i, on in enumerate(live) if on]
        c.write(layer, su.batch(cache8, live, lens), k[new].to(DEV), v[new].to(DEV))
        for s in new:
            su.ref.write(su.tables[s], lens[s] - 1, (k[s:s + 1], v[s:s + 1]))
    _same(su, layer)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_extremes(dtype):
    """Zeros, subnormals, the largest values, infinities and NaN; signed zeros keep their sign."""
    su = R.Setup(D=32, H=4, T=16, lens=[48], dtype=dtype)
    big = torch.finfo(su.dtype).max
    x = su.values(48).double()
    x[0:16, 0] = 0.0
    x[3, 0] = -0.0
    x[0:16, 1] *= 1e-7 if dtype == "fp16" else 1e-39
    x[5, 2, 7], x[6, 2, 8] = big, -big
    x[20, 0, 1], x[21, 1, 2], x[22, 2, 3] = math.inf, -math.inf, math.nan
    x[32:48, 3] = math.nan
    x[17, 3, 0] = -math.nan
    _, layer = _write_case(su, [48], [48], kv=(x.to(su.dtype), su.values(48)))
    _same(su, layer)


def test_write_step_and_other_rows_strides():
    """k and v as slices of one fused tensor; one new token each without cu_new; an idle slot writes nothing."""
    lens = [5, 0, 17, 32]
    su = R.Setup(D=128, H=4, T=16, lens=lens, dtype="bf16")
    su.fill([4, 0, 16, 31])
    c, layer = su.cache(cache8, 8), su.device_layer(cache8)
    k, v = su.values(4), su.values(4)
    fused = torch.zeros(4, 8 + 4 + 4, 128, dtype=su.dtype)
    fused[:, 8:12], fused[:, 12:] = k, v
    f = fused.to(DEV)
    c.write(layer, su.batch(cache8), f[:, 8:12], f[:, 12:])
    for s, n in enumerate(lens):
        if n:
            su.ref.write(su.tables[s], n - 1, (k[s:s + 1], v[s:s + 1]))
    _same(su, layer)


@pytest.mark.parametrize("D,T,H,by_head,dtype", [(128, 16, 8, False, "bf16"), (64, 32, 4, True, "fp16"),
                                                 (256, 5, 2, False, "fp16"), (32, 1, 1, False, "bf16"),
                                                 (32, 48, 3, True, "fp16")])
def test_read(D, T, H, by_head, dtype):
    lens, new = [1, 30, 64, 100, 0], [1, 30, 7, 51, 0]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, by_head=by_head, seed=3)
    su.fill()
    c, layer = su.cache(cache8, H), su.device_layer(cache8)
    n = sum(new)
    kv = torch.full((n, 2, H, D), 7.0, dtype=su.dtype, device=DEV)   # strided outputs
    c.read(layer, su.batch(cache8, new), kv[:, 0], kv[:, 1])
    for role in range(2):
        want = torch.cat([su.ref.tokens(role, su.tables[s], lens[s])[0][lens[s] - m:] for s, m in enumerate(new)])
        top = torch.finfo(su.dtype).max
        assert torch.equal(kv[:, role].cpu(), want.clamp(-top, top).to(su.dtype))


def test_read_saturates_and_keeps_nan():
    su = R.Setup(D=32, H=1, T=16, lens=[16], dtype="fp16")
    x = su.values(16)
    x[2, 0, 3], x[2, 0, 4], x[4, 0, 0] = 65504.0, -65504.0, math.nan
    c, layer = _write_case(su, [16], [16], kv=(x, x))
    k, v = torch.empty(16, 1, 32, dtype=su.dtype, device=DEV), torch.empty(16, 1, 32, dtype=su.dtype, device=DEV)
    c.read(layer, su.batch(cache8, [16]), k, v)
    assert k[2, 0, 3] == 65504.0 and k[2, 0, 4] == -65504.0 and torch.isnan(k[4, 0, 0])
    assert torch.isnan(k).sum() == 1


def _attend(su, lens, new, HQ, causal=True, window=0, scale=None, hints=True, c=None, layer=None, q=None, errors=None):
    c = c or su.cache(cache8, HQ)
    layer = layer or su.device_layer(cache8)
    n = sum(new) if new is not None else len(lens)
    q = su.queries(n, HQ) if q is None else q
    b = su.batch(cache8, new, lens, errors=errors, hints=hints)
    ws = torch.zeros(c.attend_workspace(b) + 1, dtype=torch.uint8, device=DEV)
    out = torch.full((n, HQ, su.D), 9.0, dtype=su.dtype, device=DEV)
    lse = torch.full((n, HQ), 9.0, device=DEV)
    c.attend(layer, b, q.to(DEV), out, lse=lse, causal=causal, window=window, scale=scale, workspace=ws)
    return q, out.cpu().double(), lse.cpu().double()


def _check(su, lens, new, q, out, lse, causal=True, window=0, scale=None):
    at = 0
    for s, n in enumerate(new if new is not None else [1] * len(lens)):
        if n == 0:
            continue
        want, wl, size, dz = su.ref.attend(su.tables[s], lens[s], q[at:at + n], causal, window, scale)
        bo, bl = R.bounds(want, wl, size, dz, su.dtype, max(1, lens[s]))
        o, x = out[at:at + n], lse[at:at + n]
        assert torch.equal(torch.isneginf(x), torch.isneginf(wl)), s
        assert torch.equal(torch.isnan(o), torch.isnan(want)), s
        f = torch.isfinite(want)
        assert bool(((o - want).abs() <= bo)[f].all()), (s, float(((o - want).abs() / bo)[f].max()))
        g = torch.isfinite(wl)
        assert bool(((x - wl).abs() <= bl)[g].all()), (s, float(((x - wl).abs() / bl)[g].max()))
        at += n


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,G,by_head,dtype", [(16, 2, 4, False, "bf16"), (32, 1, 7, True, "fp16"),
                                                 (5, 3, 1, False, "fp16"), (1, 1, 16, False, "bf16"),
                                                 (48, 2, 20, True, "bf16")])
def test_step(D, T, H, G, by_head, dtype):
    """One query a sequence: lengths 0, 1, around tiles and pages, split ranges."""
    lens = [0, 1, 2, 15, 16, 17, 63, 129, 300, 700]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, by_head=by_head, seed=D + G)
    su.fill()
    for hints in (True, False):
        q, out, lse = _attend(su, lens, None, H * G, hints=hints)
        _check(su, lens, None, q, out, lse)


@pytest.mark.parametrize("D,T,H,G,dtype", [(128, 16, 2, 4, "fp16"), (64, 24, 1, 5, "bf16"), (256, 16, 1, 2, "bf16"),
                                           (32, 5, 2, 1, "fp16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 13), (True, 64), (False, 0), (False, 40)])
def test_few_rows_masks(D, T, H, G, dtype, causal, window):
    """Drafted tokens and short chunks with every mask; idle sequences; more new tokens than held."""
    lens, new = [5, 40, 0, 130, 33, 2, 64], [5, 3, 2, 20, 0, 4, 1]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, seed=window)
    su.fill()
    q, out, lse = _attend(su, lens, new, H * G, causal, window)
    _check(su, lens, new, q, out, lse, causal, window)


@pytest.mark.parametrize("D,T,H,G,by_head,dtype", [(128, 16, 2, 4, False, "fp16"), (128, 16, 1, 7, True, "bf16"),
                                                   (64, 32, 2, 2, True, "fp16"), (256, 16, 1, 4, False, "bf16"),
                                                   (32, 16, 1, 3, False, "fp16"), (128, 24, 1, 4, False, "bf16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
def test_prompts(D, T, H, G, by_head, dtype, causal, window):
    """Whole prompts and chunks over cached tokens, ragged, next to single tokens."""
    lens, new = [200, 333, 1, 90, 150], [200, 129, 1, 1, 77]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, by_head=by_head, seed=11)
    su.fill()
    q, out, lse = _attend(su, lens, new, H * G, causal, window)
    _check(su, lens, new, q, out, lse, causal, window)


@pytest.mark.parametrize("new", [None, [4, 9, 1], [80, 30, 64]])
def test_scores_of_every_size(new):
    """Page scales far apart, scores that saturate the softmax, queries of tiny and huge magnitude."""
    lens = [90, 200, 64]
    su = R.Setup(D=64, H=2, T=16, lens=lens, dtype="bf16", seed=5, spread=4.0)
    su.fill()
    n = sum(new) if new else 3
    q = su.queries(n, 8).double()
    q[:, 0] *= 1e-30
    q[:, 1] *= 30.0
    q[:, 2] *= 2.0 ** -7
    q[:, 3] = 0.0
    q = q.to(su.dtype)
    _, out, lse = _attend(su, lens, new, 8, q=q)
    _check(su, lens, new, q, out, lse)
    _, out, lse = _attend(su, lens, new, 8, q=q, scale=0.37)
    _check(su, lens, new, q, out, lse, scale=0.37)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(2, [3, 6]), (8, [3, 6]), (4, [40, 64])])
def test_nan_reaches_only_the_rows_that_see_it(D, G, new):
    """A NaN key or value of a later token, or of one behind the window, leaves other rows as they are."""
    lens = [40, 64]
    su = R.Setup(D=D, H=1, T=16, lens=lens, dtype="fp16", seed=1)
    su.fill()
    pid, off = int(su.tables[0, 2]), 39 - 32
    su.ref.codes[1][pid, off, 0, 5] = 0x7F           # value of sequence 0's last token
    pid = int(su.tables[1, 3])
    su.ref.codes[0][pid, 62 - 48, 0, 9] = 0xFF       # key of sequence 1's last but one token
    q, out, lse = _attend(su, lens, new, G)
    _check(su, lens, new, q, out, lse)
    assert torch.isnan(out).any() and torch.isfinite(out).any()
    su.ref.codes[1][int(su.tables[1, 0]), 3, 0, 2] = 0x7F   # behind a window of 20
    q, out, lse = _attend(su, lens, new, G, window=20)
    _check(su, lens, new, q, out, lse, window=20)


def test_nan_query_stays_in_its_row():
    su = R.Setup(D=128, H=1, T=16, lens=[50], dtype="bf16")
    su.fill()
    q = su.queries(1, 4)
    q[0, 1, 7] = math.nan
    q[0, 2, 8] = math.inf
    _, out, _ = _attend(su, [50], None, 4, q=q)
    bad = torch.isnan(out).any(-1)[0].tolist()
    assert bad[1] and not bad[0] and not bad[3]


@pytest.mark.parametrize("T", [16, 24])
@pytest.mark.parametrize("op", ["write", "read", "attend", "prompt"])
def test_bad_pages(T, op):
    """Table entries that are no page, and lengths past the table: reported, skipped, nothing else touched."""
    lens, new = [60, 60, 60, 300], [60, 60, 60, 60]
    if op == "attend":
        new = [2, 1, 3, 2]
    su = R.Setup(D=64, H=2, T=T, lens=[60, 60, 60, 60], dtype="fp16", seed=2)
    su.fill()
    su.tables[1, 1] = su.pages
    su.tables[2, 0] = -5
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    if op == "write":
        c, layer = su.cache(cache8, 4), su.device_layer(cache8)
        k, v = su.values(240), su.values(240)
        c.write(layer, su.batch(cache8, new, lens, errors=errors), k.to(DEV), v.to(DEV))
        for s in range(4):
            su.ref.write(su.tables[s], lens[s] - 60, (k[60 * s:60 * s + 60], v[60 * s:60 * s + 60]))
        _same(su, layer)
    elif op == "read":
        c, layer = su.cache(cache8, 4), su.device_layer(cache8)
        k, v = (torch.full((240, 2, 64), 5.0, dtype=su.dtype, device=DEV) for _ in range(2))
        c.read(layer, su.batch(cache8, new, lens, errors=errors), k, v)
        want = torch.cat([su.ref.tokens(0, su.tables[s], lens[s])[0][lens[s] - 60:] for s in range(4)])
        assert torch.equal(k.cpu(), want.to(su.dtype))
    else:
        q, out, lse = _attend(su, lens, new, 4, errors=errors)
        _check(su, lens, new, q, out, lse)
    # sequence 3's new tokens lie past its table's row, and so does part of what its queries see
    assert errors.tolist() == [0, 1, 1, 1]


@pytest.mark.parametrize("D,T,H,G,dtype", [(64, 32, 2, 8, "fp16"), (64, 16, 1, 64, "bf16"), (32, 5, 2, 40, "bf16"),
                                           (128, 16, 4, 16, "fp16")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 13), (False, 40)])
def test_rows_on_both_sides_of_the_prompt_kernel_s_bound(D, T, H, G, dtype, causal, window):
    """Sequences of a few rows up to thousands in one batch, whichever kernel takes each."""
    lens = [100, 33, 300, 64, 0, 17, 256]
    new = [64, 13, 100, 1, 0, 17, 8]
    su = R.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, seed=G)
    su.fill()
    for hints in (True, False):
        q, out, lse = _attend(su, lens, new, H * G, causal, window, hints=hints)
        _check(su, lens, new, q, out, lse, causal, window)


@pytest.mark.parametrize("new", [[80, 30, 64], [20, 17, 60]])
def test_scores_of_every_size_with_many_heads(new):
    """Page scales far apart and queries of tiny and huge magnitude, in sequences of more than 512 rows."""
    lens = [90, 200, 64]
    su = R.Setup(D=64, H=1, T=16, lens=lens, dtype="bf16", seed=5, spread=4.0)
    su.fill()
    q = su.queries(sum(new), 32).double()
    q[:, 0:8] *= 1e-30
    q[:, 8:16] *= 30.0
    q[:, 16:24] *= 2.0 ** -7
    q[:, 24] = 0.0
    q = q.to(su.dtype)
    for scale in (None, 0.37):
        _, out, lse = _attend(su, lens, new, 32, q=q, scale=scale)
        _check(su, lens, new, q, out, lse, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_reaches_only_the_rows_that_see_it_with_many_heads(D):
    test_nan_reaches_only_the_rows_that_see_it(D, 32, [40, 64])


@pytest.mark.parametrize("T", [16, 24])
def test_bad_pages_with_many_heads(T):
    """Prompts of 960 rows whose tables hold no page, or end before the tokens."""
    lens, new = [60, 60, 60, 300], [60, 60, 60, 60]
    su = R.Setup(D=64, H=2, T=T, lens=[60, 60, 60, 60], dtype="fp16", seed=2)
    su.fill()
    su.tables[1, 1] = su.pages
    su.tables[2, 0] = -5
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    q, out, lse = _attend(su, lens, new, 32, errors=errors)
    _check(su, lens, new, q, out, lse)
    assert errors.tolist() == [0, 1, 1, 1]


def test_rows_past_the_caller_s_count_are_not_touched():
    """cu_new that promises more rows than n_new: the surplus is not read or written."""
    su = R.Setup(D=32, H=1, T=16, lens=[32, 32], dtype="fp16")
    su.fill()
    c, layer = su.cache(cache8, 1), su.device_layer(cache8)
    b = cache8.Batch(su.tables.to(DEV), torch.tensor([32, 32], dtype=torch.int32, device=DEV),
                     torch.tensor([0, 4, 900], dtype=torch.int32, device=DEV), n_new=10, max_new=6, max_len=32)
    mem = torch.full((64, 1, 32), 3.0, dtype=su.dtype, device=DEV)
    q = su.queries(10, 1).to(DEV)
    c.attend(layer, b, q, mem[:10], workspace=torch.zeros(c.attend_workspace(b) + 1, dtype=torch.uint8, device=DEV))
    c.read(layer, b, mem[20:30], mem[40:50])
    rest = torch.cat([mem[10:20], mem[30:40], mem[50:]])
    assert bool((rest == 3.0).all()) and not bool((mem[:10] == 3.0).all(-1).any())


@pytest.mark.parametrize("new", [None, [130, 40, 300]])
def test_same_result_every_time_and_on_another_stream(new):
    lens = [5000, 300, 1200]
    su = R.Setup(D=128, H=2, T=16, lens=lens, dtype="bf16")
    c = su.cache(cache8, 8)
    layer = cache8.Layer(*(torch.randint(0, 126, (su.pages, 16, 2, 128), dtype=torch.uint8, device=DEV) for _ in range(2)),
                         *(torch.full((su.pages, 2), 2.0 ** -7, device=DEV) for _ in range(2)))
    n = sum(new) if new else 3
    q = su.queries(n, 8).to(DEV)
    b = su.batch(cache8, new, lens)
    ws = torch.zeros(c.attend_workspace(b) + 1, dtype=torch.uint8, device=DEV)
    outs = []
    side = torch.cuda.Stream()
    for i in range(6):
        out = torch.empty(n, 8, 128, dtype=su.dtype, device=DEV)
        lse = torch.empty(n, 8, device=DEV)
        torch.cuda.synchronize()
        c.attend(layer, b, q, out, lse=lse, workspace=ws, stream=side if i % 2 else None)
        torch.cuda.synchronize()
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    # the workspace is left as the next call wants it: another batch on it gives what a fresh one gives
    b2 = su.batch(cache8, None, [700, 5000, 64])
    r = []
    for w in (ws, torch.zeros_like(ws)):
        out = torch.empty(3, 8, 128, dtype=su.dtype, device=DEV)
        c.attend(layer, b2, q[:3], out, workspace=w)
        r.append(out)
    assert torch.equal(*r)


def test_captured_step_with_other_lengths():
    """A captured write + attend, replayed after the lengths, tables and inputs in its arrays changed."""
    lens = [20, 47, 1]
    su = R.Setup(D=128, H=2, T=16, lens=[90, 90, 90], dtype="bf16", seed=9)
    su.fill([19, 46, 0])
    c, layer = su.cache(cache8, 8), su.device_layer(cache8)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    b = cache8.Batch(su.tables.to(DEV), dl, max_new=1, max_len=90)
    k, v = (torch.zeros(3, 2, 128, dtype=su.dtype, device=DEV) for _ in range(2))
    q = torch.zeros(3, 8, 128, dtype=su.dtype, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(3, 8, device=DEV)
    ws = torch.zeros(c.attend_workspace(b) + 1, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    warm = su.device_layer(cache8)
    c.write(warm, b, k, v)
    c.attend(warm, b, q, out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.write(layer, b, k, v)
        c.attend(layer, b, q, out, lse=lse, workspace=ws)
    for step in range(30):
        nk, nv, nq = su.values(3), su.values(3), su.queries(3, 8)
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        for s in range(3):
            su.ref.write(su.tables[s], lens[s] - 1, (nk[s:s + 1], nv[s:s + 1]))
        _check(su, lens, None, nq, out.cpu().double(), lse.cpu().double())
        lens = [n + 1 for n in lens]
    _same(su, layer)


def test_offsets_past_32_bits():
    """Pages beyond 2^32 bytes of codes."""
    H, T, D = 8, 64, 256
    pages = (1 << 32) // (H * T * D) + 20
    su = R.Setup(D=D, H=H, T=T, lens=[100], dtype="fp16")
    c = cache8.Cache8(dtype="fp16", head_dim=D, num_kv_heads=H, num_q_heads=2 * H, block_tokens=T, num_blocks=pages)
    layer = c.new_layer()
    high = [pages - 1, pages - 9]
    tables = torch.tensor([high], dtype=torch.int32, device=DEV)
    k, v, q = su.values(100), su.values(100), su.queries(100, 2 * H)
    cu = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    lens = torch.tensor([100], dtype=torch.int32, device=DEV)
    b = cache8.Batch(tables, lens, cu, n_new=100, max_new=100, max_len=100)
    c.write(layer, b, k.to(DEV), v.to(DEV))
    su.ref.write(su.tables[0], 0, (k, v))
    back = [torch.empty(100, H, D, dtype=su.dtype, device=DEV) for _ in range(2)]
    c.read(layer, b, *back)
    for role in range(2):
        assert torch.equal(back[role].cpu().double(), su.ref.tokens(role, su.tables[0], 100)[0])
    for rows in (100, 1):
        bb = b if rows == 100 else cache8.Batch(tables, lens, max_len=100)
        out, lse = torch.empty(rows, 2 * H, D, dtype=su.dtype, device=DEV), torch.empty(rows, 2 * H, device=DEV)
        ws = torch.zeros(c.attend_workspace(bb) + 1, dtype=torch.uint8, device=DEV)
        c.attend(layer, bb, q[:rows].to(DEV), out, lse=lse, workspace=ws)
        _check(su, [100], [rows], q[:rows], out.cpu().double(), lse.cpu().double())
    assert int(layer.k.view(pages, -1)[:pages - 9].count_nonzero()) == 0


def test_refusals():
    su = R.Setup(D=64, H=2, T=16, lens=[600], dtype="fp16")
    c, layer = su.cache(cache8, 4), su.device_layer(cache8)
    b = su.batch(cache8)
    kv, q = su.values(1).to(DEV), su.queries(1, 4).to(DEV)
    out = torch.empty_like(q)
    ws = torch.zeros(c.attend_workspace(b), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0

    def code(f):
        with pytest.raises(cache8.KvCodecError) as e:
            f()
        return e.value.code

    assert code(lambda: c.attend(layer, b, q, out)) == -1                          # workspace missing
    assert code(lambda: c.attend(layer, b, q, out, workspace=ws[:-16])) == -1      # too small
    odd = torch.zeros(ws.numel() + 16, dtype=torch.uint8, device=DEV)[4:]
    assert code(lambda: c.attend(layer, b, q, out, workspace=odd)) == -5
    big = torch.zeros(3, 4, 68, dtype=su.dtype, device=DEV)
    assert code(lambda: c.write(layer, b, big[:1, :2, 4:], kv)) == -5              # rows not 16-byte aligned
    narrow = torch.zeros(1, 4 * 64, dtype=su.dtype, device=DEV)
    assert code(lambda: c.attend(layer, b, q, narrow.as_strided((1, 4, 64), (256, 32, 1)), workspace=ws)) == -3
    bad = cache8._Rows(torch.zeros(64).data_ptr() & ~15, 128, 64)                  # pageable host memory
    import ctypes as C
    rc = cache8.lib().kv_cache8_write(c._h, layer._ref, b._ref, C.addressof(bad), C.addressof(bad), None)
    assert rc == -9
    for f in (lambda: c.write(layer, b, kv.float(), kv), lambda: c.write(layer, b, kv[:, :1], kv),
              lambda: c.write(layer, b, kv.cpu(), kv), lambda: c.attend(layer, b, kv, out, workspace=ws),
              lambda: c.attend(layer, b, q, out, lse=torch.empty(1, 3, device=DEV), workspace=ws),
              lambda: c.attend(layer, b, q, out, scale=-1.0, workspace=ws),
              lambda: c.attend(layer, b, q, out, window=-1, workspace=ws),
              lambda: c.write(cache8.Layer(layer.k[:-1], layer.v, layer.k_scale[:-1], layer.v_scale), b, kv, kv),
              lambda: cache8.Batch(b.tables.long(), b.lens), lambda: cache8.Batch(b.tables, b.lens.cpu())):
        with pytest.raises(ValueError):
            f()
    # no rows: nothing is launched
    empty = cache8.Batch(torch.zeros(0, 4, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    none = torch.empty(0, 4, 64, dtype=su.dtype, device=DEV)
    c.attend(layer, empty, none, none)


def test_the_example_serves_and_offloads():
    """examples/serve_cache8.py end to end, small; ."""
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("serve_cache8", os.path.join(root, "examples", "serve_cache8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.serve(3, 90, 20)
    assert not r["errors"].any() and r["encoded"] == r["segments"] == 2 * 7 and r["tokens"] == 110
    assert torch.isfinite(r["out"].float()).all() and torch.isfinite(r["step_out"].float()).all()
    assert torch.equal(r["pages"].view(2, -1, 8, 128)[:, 110:], torch.zeros_like(r["pages"].view(2, -1, 8, 128)[:, 110:]))
