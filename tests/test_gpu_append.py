"""Appending with the position rotation to 16-bit and to 8-bit pages on the GPU: bit for bit what the stated FP32
operations give, and within a rounding of the rotation in 64 bits."""
import math

import pytest
import torch

import cache8_ref as R8
import cache16_ref as R
from kv_cache_page_gb300 import cache8, cache16

pytestmark = pytest.mark.gpu
DEV = "cuda"
POSITIONS = 400


def _rotation(dim, neighbours=False, positions=POSITIONS, split=True):
    """(cos, sin) on the CPU and the device's rotation; split: the two halves of one table."""
    c, s = R.tables(positions, dim)
    if split:
        both = torch.cat([c, s], 1).to(DEV)
        return (c, s), cache8.Rotation(both[:, :dim // 2], both[:, dim // 2:], interleaved=neighbours)
    return (c, s), cache8.Rotation(c.to(DEV), s.to(DEV), interleaved=neighbours)


def _rows(lens, new):
    """Sequence and position of each row."""
    return [(s, lens[s] - c + i) for s, c in enumerate(new if new is not None else [1] * len(lens)) for i in range(c)]


def _fused(su, n, HQ):
    """k, v and q of n rows as one projection leaves them (views of one tensor), and on the CPU."""
    k, v, q = su.values(n), su.values(n), su.values(n, HQ)
    if n and HQ > 1:
        q[0, 0, :8], k[0, 0, 8:16] = 0.0, -0.0
    f = torch.cat([q, k, v], 1).to(DEV)
    return (k, v, q), (f[:, HQ:HQ + su.H], f[:, HQ + su.H:], f[:, :HQ])


def _turned(x, rows, tab, neighbours):
    return R.turn(x.float(), [p for _, p in rows], *tab, neighbours)


def _queries_want(q, rows, tab, neighbours, dtype):
    """round(FP32 rotation), 0 without a position; what is not turned as it is."""
    want = _turned(q, rows, tab, neighbours).to(dtype)
    none = torch.tensor([p < 0 for _, p in rows])
    return torch.where(none[:, None, None], torch.zeros((), dtype=dtype), want)


def _near(got, x, rows, tab, neighbours):
    """Within the rounding to the type and the FP32 roundings (two products, a sum) of the rotation in 64 bits."""
    want = R.turn(x.double(), [p for _, p in rows], *tab, neighbours)
    size = R.turn(x.double().abs(), [p for _, p in rows], tab[0].abs(), -tab[1].abs(), neighbours).abs() + x.double().abs()
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    most = want.abs() * torch.finfo(got.dtype).eps / 2 * (1 + 1e-6) + size * 2 * 3 * 2.0 ** -24 + tiny
    ok = torch.isfinite(want)
    assert bool(((got.double() - want).abs() <= most)[ok].all())


def _same_bits(got, want):
    """Equal bit for bit, NaN anywhere equal to NaN."""
    a, b = torch.isnan(got.float()), torch.isnan(want.float())
    view = torch.int16 if got.element_size() == 2 else torch.uint8
    off = (a != b) | (~a & (got.contiguous().view(view) != want.contiguous().view(view)))
    where = off.nonzero()
    at = tuple(where[0].tolist()) if len(where) else ()
    assert not len(where), (len(where), off.numel(), at, float(got[at]), float(want[at]))


def _append16(su, lens, new, HQ, R_dim, neighbours=False, queries=True, tab=None, rotation=None, errors=None):
    c, layer = su.cache(cache16, HQ), su.device_layer(cache16)
    b = su.batch(cache8, new, lens, errors=errors)
    rows = _rows(lens, new)
    (k, v, q), (kd, vd, qd) = _fused(su, len(rows), HQ)
    if rotation is None and R_dim:
        tab, rotation = _rotation(R_dim, neighbours)
    qo = torch.full((len(rows), HQ, su.D), 9.0, dtype=su.dtype, device=DEV) if queries else None
    c.append(layer, b, kd, vd, rotation=rotation, q=qd if queries else None, q_out=qo)
    turned = _turned(k, rows, tab, neighbours).to(su.dtype) if R_dim else k
    for i, (s, p) in enumerate(rows):
        su.put(s, p, turned[i:i + 1], v[i:i + 1])
    for got, want in zip(su.bits_of(layer), su.pool):
        _same_bits(got.view(su.dtype), want)
    if queries:
        _same_bits(qo.cpu(), _queries_want(q, rows, tab, neighbours, su.dtype))
        some = [i for i, (_, p) in enumerate(rows) if 0 <= p < tab[0].shape[0]]
        _near(qo.cpu()[some], q[some], [rows[i] for i in some], tab, neighbours)
    return c, layer


NEW = [1, 0, 3, 40, 17, 1, 64, 1, 5]
LENS = [1, 7, 3, 61, 33, 17, 64, 64, 2]     # the last: more new tokens than held


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,G,layout,dtype", [(16, 8, 4, "nhd", "bf16"), (32, 2, 5, "hnd", "fp16"), (5, 3, 1, "packed", "fp16"),
                                                (1, 1, 16, "nhd", "bf16"), (130, 1, 1, "packed", "bf16")])
@pytest.mark.parametrize("part,neighbours", [(1, False), (1, True), (2, False), (2, True)])
def test_append16(D, T, H, G, layout, dtype, part, neighbours):
    """Ragged chunks, single tokens, none; all channels turned or a half; every layout; nothing else is touched."""
    su = R.Setup(D=D, H=H, T=T, lens=LENS, dtype=dtype, layout=layout, seed=D + T)
    su.fill([max(0, n - c) for n, c in zip(LENS, NEW)])
    _append16(su, LENS, NEW, H * G, max(16, D // part), neighbours)


@pytest.mark.parametrize("R_dim", [0, 16, 48, 80, 96, 112, 128])
@pytest.mark.parametrize("neighbours", [False, True])
def test_append16_some_channels(R_dim, neighbours):
    su = R.Setup(D=128, H=3, T=16, lens=LENS, dtype="bf16", seed=R_dim)
    _append16(su, LENS, NEW, 6, R_dim, neighbours, queries=R_dim > 0)


@pytest.mark.parametrize("H,D,dtype", [(8, 128, "bf16"), (1, 32, "fp16"), (5, 64, "fp16")])
def test_append16_step(H, D, dtype):
    """One token a sequence without cu_new, idle slots among them."""
    lens = [5, 0, 17, 32, 1, 300, 0, 16] * 5
    su = R.Setup(D=D, H=H, T=16, lens=lens, dtype=dtype)
    su.fill([max(0, n - 1) for n in lens])
    _append16(su, lens, None, 2 * H, D)


def test_append16_many_short_sequences():
    """Several rows, and so several sequences, to a warp; empty sequences between them."""
    lens = [(7 * i) % 23 for i in range(700)]
    new = [min(n, (3 * i) % 5) if i % 4 else 0 for i, n in enumerate(lens)]
    su = R.Setup(D=32, H=1, T=8, lens=lens, dtype="fp16")
    _append16(su, lens, new, 1, 32)
    _append16(su, lens, new, 1, 16, True)


@pytest.mark.parametrize("neighbours", [False, True])
def test_queries_in_place(neighbours):
    su = R.Setup(D=64, H=2, T=16, lens=[40, 9], dtype="bf16")
    c, layer = su.cache(cache16, 6), su.device_layer(cache16)
    tab, rotation = _rotation(48, neighbours, split=False)
    rows = _rows([40, 9], [40, 9])
    (k, v, q), (kd, vd, qd) = _fused(su, 49, 6)
    c.append(layer, su.batch(cache8, [40, 9]), kd, vd, rotation=rotation, q=qd, q_out=qd)
    _same_bits(qd.cpu(), _queries_want(q, rows, tab, neighbours, su.dtype))
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


@pytest.mark.parametrize("eight", [False, True])
def test_positions_past_the_table_and_bad_pages(eight):
    """NaN keys and queries, nothing else; what has no page is not written; both are reported."""
    lens, new = [60, 60, 60, 30], [60, 5, 60, 30]
    errors = torch.zeros(4, dtype=torch.int32, device=DEV)
    tab, rotation = _rotation(64, positions=50)
    if not eight:
        su = R.Setup(D=64, H=2, T=16, lens=lens, dtype="fp16", seed=2)
        su.tables[2, 1] = su.pages + 7
        _append16(su, lens, new, 4, 64, tab=tab, rotation=rotation, errors=errors)
    else:
        su = R8.Setup(D=64, H=2, T=16, lens=lens, dtype="fp16", seed=2)
        su.fill([0, 55, 0, 0])
        su.tables[2, 1] = su.pages + 7
        _append8(su, lens, new, 4, 64, tab=tab, rotation=rotation, errors=errors)
    assert errors.tolist() == [4, 4, 5, 0]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
def test_positions_past_the_table_keep_what_is_not_turned(eight, neighbours):
    """NaN in the turned channels alone."""
    lens, new = [60, 55], [60, 5]
    errors = torch.zeros(2, dtype=torch.int32, device=DEV)
    tab, rotation = _rotation(48, neighbours, positions=50)
    module, append = (R8, _append8) if eight else (R, _append16)
    su = module.Setup(D=64, H=2, T=16, lens=lens, dtype="bf16", seed=2)
    su.fill([0, 50])
    append(su, lens, new, 4, 48, neighbours, tab=tab, rotation=rotation, errors=errors)
    assert errors.tolist() == [4, 4]


def test_signed_zeros_and_what_is_no_number():
    """Infinities and NaN stay in their pair and row; channels that are not turned keep their bits."""
    su = R.Setup(D=64, H=1, T=16, lens=[16], dtype="fp16")
    c, layer = su.cache(cache16, 1), su.device_layer(cache16)
    tab, rotation = _rotation(32)
    k, v = su.values(16), su.values(16)
    k[3, 0, 2], k[4, 0, 18], k[5, 0, 40], k[6] = math.inf, math.nan, math.nan, 0.0
    k[7] = -k[6]
    k[5].view(torch.int16)[0, 41] = 0x7c01      # a NaN of other bits
    c.append(layer, su.batch(cache8, [16]), k.to(DEV), v.to(DEV), rotation=rotation)
    turned = _turned(k, _rows([16], [16]), tab, False).to(su.dtype)
    turned[..., 32:] = k[..., 32:]
    su.put(0, 0, turned, v)
    got = su.bits_of(layer)
    _same_bits(got[0].view(su.dtype), su.pool[0])
    assert int(got[0][int(su.tables[0, 0]), 5, 0, 41]) == 0x7c01 and torch.equal(got[1], su.pool[1].view(torch.int16))


# ---------------------------------------------------------------- 8 bits
def _append8(su, lens, new, HQ, R_dim, neighbours=False, queries=True, tab=None, rotation=None, errors=None, kv=None):
    c, layer = su.cache(cache8, HQ), su.device_layer(cache8)
    b = su.batch(cache8, new, lens, errors=errors)
    rows = _rows(lens, new)
    (k, v), q = kv or (su.values(len(rows)), su.values(len(rows))), su.queries(len(rows), HQ)
    if rotation is None:
        tab, rotation = _rotation(R_dim, neighbours)
    qo = torch.full((len(rows), HQ, su.D), 9.0, dtype=su.dtype, device=DEV)
    c.append(layer, b, k.to(DEV), v.to(DEV), rotation=rotation, q=q.to(DEV) if queries else None, q_out=qo if queries else None)
    turned = _turned(k, rows, tab, neighbours)
    at = 0
    for s, n in enumerate(new if new is not None else [1] * len(lens)):
        su.ref.write(su.tables[s], lens[s] - n, (turned[at:at + n], v[at:at + n]))
        at += n
    for role, codes in enumerate(su.codes_of(layer)):
        _same_bits(codes.view(torch.float8_e4m3fn), su.ref.codes[role].view(torch.float8_e4m3fn))
        got = (layer.k_scale, layer.v_scale)[role].cpu().double()
        assert torch.equal(torch.nan_to_num(got, nan=-1), torch.nan_to_num(su.ref.scale[role], nan=-1)), role
    if queries:
        _same_bits(qo.cpu(), _queries_want(q, rows, tab, neighbours, su.dtype))
    return c, layer


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,G,by_head,dtype", [(16, 8, 4, False, "bf16"), (32, 2, 5, True, "fp16"), (5, 3, 1, False, "fp16"),
                                                 (1, 1, 16, True, "bf16"), (130, 1, 1, False, "bf16")])
@pytest.mark.parametrize("part,neighbours", [(1, False), (1, True), (2, False), (2, True)])
def test_append8(D, T, H, G, by_head, dtype, part, neighbours):
    """Codes and scales bit for bit: fresh pages, half-filled pages whose scale stays or grows, one token, none."""
    new = [1, 0, 3, 40, 17, 1, 2 * T, 1]
    lens = [1, 7, 3, 61, 33, T + 1, 2 * T, 2 * T]
    su = R8.Setup(D=D, H=H, T=T, lens=lens, dtype=dtype, by_head=by_head, seed=D + T)
    su.fill([n - c for n, c in zip(lens, new)])
    _append8(su, lens, new, H * G, max(16, D // part), neighbours)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append8_extremes(dtype):
    """Zeros, subnormals, the largest values (which the rotation takes past the type), infinities and NaN."""
    su = R8.Setup(D=32, H=4, T=16, lens=[48], dtype=dtype)
    big = torch.finfo(su.dtype).max
    x = su.values(48).double()
    x[0:16, 0] = 0.0
    x[3, 0] = -0.0
    x[0:16, 1] *= 1e-7 if dtype == "fp16" else 1e-39
    x[5, 2, 7], x[5, 2, 23], x[6, 2, 8] = big, -big, -big
    x[20, 0, 1], x[21, 1, 2], x[22, 2, 3] = math.inf, -math.inf, math.nan
    x[32:48, 3] = math.nan
    _append8(su, [48], [48], 4, 32, kv=(x.to(su.dtype), su.values(48)))


def test_append8_without_a_rotation_is_write():
    lens, new = [40, 9, 64], [40, 1, 3]
    su = R8.Setup(D=64, H=2, T=16, lens=lens, dtype="bf16", seed=3)
    su.fill([0, 8, 61])
    c, layers = su.cache(cache8, 4), [su.device_layer(cache8) for _ in range(2)]
    k, v, b = su.values(44).to(DEV), su.values(44).to(DEV), su.batch(cache8, new)
    c.write(layers[0], b, k, v)
    c.append(layers[1], b, k, v, rotation=None)
    for name in ("k", "v", "k_scale", "v_scale"):
        a, o = (getattr(y, name) for y in layers)
        assert torch.equal(a.view(torch.uint8), o.view(torch.uint8)), name


def test_a_table_of_no_turn_writes_what_write_does():
    """cos 1 and sin 0: the FP32 way through append and the 16-bit way through write agree bit for bit."""
    lens, new = [200, 9, 64], [200, 1, 33]
    for dtype in ("fp16", "bf16"):
        su = R8.Setup(D=128, H=2, T=16, lens=lens, dtype=dtype, seed=3)
        su.fill([0, 8, 31])
        c, layers = su.cache(cache8, 4), [su.device_layer(cache8) for _ in range(2)]
        k, v, b = su.values(234).to(DEV), su.values(234).to(DEV), su.batch(cache8, new)
        one = torch.ones(200, 64, device=DEV)
        c.write(layers[0], b, k, v)
        c.append(layers[1], b, k, v, rotation=cache8.Rotation(one, torch.zeros_like(one)))
        for name in ("k", "v", "k_scale", "v_scale"):
            a, o = (getattr(y, name) for y in layers)
            assert torch.equal(a.view(torch.uint8), o.view(torch.uint8)), name


# ---------------------------------------------------------------- both
@pytest.mark.parametrize("eight", [False, True])
def test_rows_past_the_caller_s_count_are_not_touched(eight):
    """cu_new that promises more rows than n_new: the surplus is not read or written."""
    c = (cache8.Cache8 if eight else cache16.Cache16)(dtype="fp16", head_dim=32, num_kv_heads=1, num_q_heads=1, block_tokens=16,
                                                      num_blocks=6)
    layer = c.new_layer()
    tables = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    b = cache8.Batch(tables, torch.tensor([32, 32], dtype=torch.int32, device=DEV),
                     torch.tensor([0, 4, 900], dtype=torch.int32, device=DEV), n_new=10, max_new=6, max_len=32)
    mem = torch.full((64, 1, 32), 3.0, dtype=torch.float16, device=DEV)
    _, rotation = _rotation(32)
    c.append(layer, b, mem[20:30], mem[20:30], rotation=rotation, q=mem[30:40], q_out=mem[:10])
    assert bool((mem[10:] == 3.0).all()) and not bool((mem[:10] == 3.0).all(-1).any())
    held = (layer.v.view(6, 16, 32) != 0).any(-1)
    assert held.sum() == 10 and bool(held[1, 12:].all()) and bool(held[3, 10:].all())


@pytest.mark.parametrize("eight", [False, True])
def test_captured_step_with_other_lengths_and_streams(eight):
    """A captured append and attention, replayed after lengths, tables and inputs in its arrays changed."""
    lens, HQ = [20, 47, 1], 8
    if eight:
        su = R8.Setup(D=128, H=2, T=16, lens=[90] * 3, dtype="bf16", seed=9)
        module = cache8
    else:
        su = R.Setup(D=128, H=2, T=16, lens=[90] * 3, dtype="bf16", seed=9)
        module = cache16
    su.fill([19, 46, 0])
    c, layer, warm = su.cache(module, HQ), su.device_layer(module), su.device_layer(module)
    tab, rotation = _rotation(128)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    b = cache8.Batch(su.tables.to(DEV), dl, max_new=1, max_len=90)
    k, v = (torch.zeros(3, 2, 128, dtype=su.dtype, device=DEV) for _ in range(2))
    q = torch.zeros(3, HQ, 128, dtype=su.dtype, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(3, HQ, device=DEV)
    ws = torch.zeros(c.attend_workspace(b) + 16, dtype=torch.uint8, device=DEV)

    def step(y):
        c.append(y, b, k, v, rotation=rotation, q=q, q_out=q)
        c.attend(y, b, q, out, lse=lse, workspace=ws)

    step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(layer)
    from test_gpu_cache16 import _check as check16
    from test_gpu_cache8 import _check as check8
    for i in range(30):
        nk, nv, nq = su.values(3), su.values(3), torch.randn(3, HQ, 128, generator=su.g).to(su.dtype)
        k.copy_(nk), v.copy_(nv), q.copy_(nq)
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        rows = _rows(lens, None)
        turned = _turned(nk, rows, tab, False)
        for s in range(3):
            if eight:
                su.ref.write(su.tables[s], lens[s] - 1, (turned[s:s + 1], nv[s:s + 1]))
            else:
                su.put(s, lens[s] - 1, turned[s:s + 1].to(su.dtype), nv[s:s + 1])
        got = q.cpu()
        _same_bits(got, _queries_want(nq, rows, tab, False, su.dtype))
        (check8 if eight else check16)(su, lens, None, got, out.cpu().double(), lse.cpu().double())
        lens = [n + 1 for n in lens]


@pytest.mark.parametrize("eight", [False, True])
def test_offsets_past_32_bits(eight):
    """Pages beyond 2^32 bytes of K."""
    H, T, D = 8, 64, 256
    pages = (1 << 32) // (H * T * D * (1 if eight else 2)) + 20
    c = (cache8.Cache8 if eight else cache16.Cache16)(dtype="fp16", head_dim=D, num_kv_heads=H, num_q_heads=H, block_tokens=T,
                                                      num_blocks=pages)
    layer = c.new_layer()
    high = [pages - 1, pages - 9]
    su = R.Setup(D=D, H=H, T=T, lens=[100], dtype="fp16")
    k, v = su.values(100), su.values(100)
    b = cache8.Batch(torch.tensor([high], dtype=torch.int32, device=DEV), torch.tensor([100], dtype=torch.int32, device=DEV),
                     torch.tensor([0, 100], dtype=torch.int32, device=DEV), n_new=100, max_new=100, max_len=100)
    tab, rotation = _rotation(D)
    c.append(layer, b, k.to(DEV), v.to(DEV), rotation=rotation)
    turned = _turned(k, _rows([100], [100]), tab, False)
    if eight:
        ref = R8.Cache(2, T, H, D)
        ref.write([0, 1], 0, (turned, v))
        for mem, want in ((layer.k, ref.codes[0]), (layer.v, ref.codes[1])):
            got = mem.view(pages, T, H, D)[high].cpu()
            assert torch.equal(got.view(-1, H, D)[:100], want.view(-1, H, D)[:100])
    else:
        for mem, want in ((layer.k, turned.half()), (layer.v, v)):
            assert torch.equal(mem.view(pages, T, H, D)[high].cpu().view(-1, H, D)[:100], want)
    assert int(layer.k.view(pages, -1)[:pages - 9].count_nonzero()) == 0


@pytest.mark.parametrize("eight", [False, True])
def test_refusals(eight):
    c = (cache8.Cache8 if eight else cache16.Cache16)(dtype="fp16", head_dim=64, num_kv_heads=2, num_q_heads=4, block_tokens=16,
                                                      num_blocks=4)
    layer = c.new_layer()
    b = cache8.Batch(torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV))
    kv, q = torch.zeros(1, 2, 64, dtype=torch.float16, device=DEV), torch.zeros(1, 4, 64, dtype=torch.float16, device=DEV)
    _, rot = _rotation(64)

    def code(rotation, q=None, q_out=None):
        with pytest.raises(cache8.KvCodecError) as e:
            c.append(layer, b, kv, kv, rotation=rotation, q=q, q_out=q_out)
        return e.value.code

    wide = torch.zeros(50, 200, device=DEV)
    turn = lambda lo, hi, cls=cache8.Rotation: cls(wide[:, lo:hi], wide[:, lo:hi])  # noqa: E731
    assert code(turn(0, 36)) == -1                       # 72 channels: no multiple of 16
    assert code(turn(0, 40)) == -1                       # 80 channels of 64
    assert code(turn(2, 34)) == -5                       # not 16-byte aligned
    odd = torch.zeros(50, 33, device=DEV)[:, :32]
    assert code(cache8.Rotation(odd, odd)) == -5         # rows not 16-byte aligned
    over = torch.zeros(4, 64, device=DEV).as_strided((4, 32), (16, 1))
    assert code(cache8.Rotation(over, over)) == -3       # rows overlap
    narrow = torch.zeros(1, 4 * 64, dtype=torch.float16, device=DEV).as_strided((1, 4, 64), (256, 32, 1))
    assert code(rot, q, narrow) == -3
    for f in (lambda: c.append(layer, b, kv, kv, rotation=rot, q=q), lambda: c.append(layer, b, kv, kv, rotation=None, q=q, q_out=q),
              lambda: c.append(layer, b, kv, q, rotation=rot), lambda: c.append(layer, b, kv.float(), kv, rotation=rot),
              lambda: c.append(layer, b, kv, kv, rotation=rot, q=kv, q_out=kv),
              lambda: cache8.Rotation(wide.double(), wide.double()), lambda: cache8.Rotation(wide, wide[1:]),
              lambda: cache8.Rotation(wide.cpu(), wide.cpu()), lambda: cache8.Rotation(wide[:, ::2], wide[:, ::2]),
              lambda: cache8.Rotation(wide[:, :32], wide[:, :32].contiguous()), lambda: cache8.Rotation(wide[0], wide[0])):
        with pytest.raises(ValueError):
            f()
    assert int(layer.k.count_nonzero()) == 0
    empty = cache8.Batch(torch.zeros(0, 4, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV))
    none = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    c.append(layer, empty, none, none, rotation=rot)


def test_the_table_of_angles():
    """Rotation.of in 64 bits: the angles of far positions are right to FP32."""
    r = cache8.Rotation.of(64, 200001, theta=1e4)
    for p in (0, 1, 777, 200000):
        for i in (0, 1, 5, 31):
            a = p * 1e4 ** (-2 * i / 64)
            assert abs(float(r.cos[p, i]) - math.cos(a)) < 2.0 ** -24 + 1e-9 and abs(float(r.sin[p, i]) - math.sin(a)) < 2.0 ** -24 + 1e-9
