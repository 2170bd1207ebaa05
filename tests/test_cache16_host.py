"""Host-only checks of the live 16-bit cache and of the rotation (no GPU): exports, structures, refusals, workspace
sizes; and the reference that the GPU tests use."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import cache16_ref as R
from kv_cache_page_gb300 import build as kbuild
from kv_cache_page_gb300 import cache8, cache16

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "kv_cache16.h")).read()
    names = set(re.findall(r"^\s*\w+\s+(kv_cache16_\w+)\s*\(", text, re.M))
    assert names == set(cache16.EXPORTS)
    for lib in (cache16.lib(), C.CDLL(kbuild.build(debug=True))):
        for n in names:
            assert hasattr(lib, n), n
    assert cache16.lib().kv_cache16_abi_version() == cache16.ABI_VERSION


def test_constants_and_structure_sizes():
    text = open(os.path.join(ROOT, "include", "kv_cache8.h")).read()
    bits = {n: int(v) for n, v in re.findall(r"^#define KV_CACHE8_(BAD_POSITION|NEIGHBOURS) (\d+)u", text, re.M)}
    assert bits == {"BAD_POSITION": cache8.BAD_POSITION, "NEIGHBOURS": cache8.NEIGHBOURS}
    assert C.sizeof(cache8._Rotation) == 40 and C.sizeof(cache16._Layer) == 16


def _kw(**over):
    kw = dict(dtype="bf16", head_dim=128, num_kv_heads=8, num_q_heads=32, block_tokens=16, num_blocks=64)
    kw.update(over)
    return kw


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), -2),
    (dict(head_dim=16), -2),
    (dict(num_kv_heads=0), -1),
    (dict(num_q_heads=12), -1),
    (dict(num_q_heads=8 * 65), -1),
    (dict(block_tokens=0), -1),
    (dict(block_tokens=32769), -1),
    (dict(num_blocks=0), -1),
    (dict(num_blocks=1 << 31), -1),
    (dict(geometry_overrides={"dtype": 3}), -1),
    (dict(geometry_overrides={"reserved": 1}), -1),
    (dict(geometry_overrides={"abi_version": 2}), -7),
    (dict(geometry_overrides={"struct_size": 56}), -7),
    (dict(strides=(16 * 8 * 128, 8 * 128, 124)), -5),
    (dict(strides=(16 * 8 * 128, 8 * 128, 64)), -3),     # heads overlap
    (dict(strides=(8 * 128, 8 * 128, 128)), -3),         # pages overlap
    (dict(strides=(16 * 8 * 128, 0, 128)), -3),
    (dict(strides=(1 << 62, 8 * 128, 128), num_blocks=1), -3),   # no offset in bytes
])
def test_geometry_refusals(over, code):
    with pytest.raises(cache16.KvCodecError) as e:
        cache16.Cache16(**_kw(**over))
    assert e.value.code == code


def test_accepted_layouts():
    cache16.Cache16(**_kw()).close()
    cache16.Cache16(**_kw(strides=(16 * 8 * 128, 128, 16 * 128))).close()              # pages by head
    cache16.Cache16(**_kw(strides=(2 * 16 * 8 * 128, 256, 2 * 16 * 128))).close()      # packed
    cache16.Cache16(**_kw(num_blocks=1, num_kv_heads=1, num_q_heads=5, strides=(8, 128, 8))).close()
    cache16.Cache16(**_kw(block_tokens=1, strides=(1024, 1024, 128))).close()


def _batch(**over):
    b = dict(struct_size=64, n_seqs=4, n_new=4, max_new=1, max_len=1000, table_width=80, table_stride=80)
    b.update(over)
    return cache8._Batch(**b)


def _workspace(cache, b):
    n = C.c_uint64()
    return cache16.lib().kv_cache16_attend_workspace(cache._h, C.byref(b), C.byref(n)), n.value


@pytest.mark.parametrize("over,code", [
    (dict(struct_size=56), -7),
    (dict(n_seqs=65536, n_new=65536), -1),
    (dict(n_new=5), -1),                           # one new token each without cu_new
    (dict(n_seqs=0, n_new=3, cu_new=64), -1),
    (dict(n_new=1 << 30, cu_new=64), -1),          # rows past 31 bits
])
def test_batch_refusals(over, code):
    assert _workspace(cache16.Cache16(**_kw()), _batch(**over))[0] == code


def test_one_workspace_size_for_every_batch():
    c = cache16.Cache16(**_kw())
    sizes = {_workspace(c, _batch(**o)) for o in (dict(), dict(n_seqs=1, n_new=1, max_len=131072), dict(n_new=900, cu_new=64),
                                                   dict(max_len=0, table_width=1), dict(max_new=0))}
    assert len(sizes) == 1 and sizes.pop()[0] == 0
    assert _workspace(c, _batch(n_seqs=0, n_new=0)) == (0, 0)


def test_null_arguments():
    L, n = cache16.lib(), C.c_uint64()
    c = cache16.Cache16(**_kw())
    b, y = _batch(lens=64, tables=64), cache16._Layer(0, 0)
    r = cache8._Rows(0, 1024, 128)
    ref = C.addressof
    assert L.kv_cache16_create(None, C.byref(C.c_void_p())) == -1
    assert L.kv_cache16_destroy(None) == -1
    assert L.kv_cache16_attend_workspace(c._h, None, C.byref(n)) == -1
    assert L.kv_cache16_attend_workspace(c._h, ref(b), None) == -1
    assert L.kv_cache16_append(None, ref(y), ref(b), ref(r), ref(r), None, None, None, None) == -1
    assert L.kv_cache16_append(c._h, ref(y), None, ref(r), ref(r), None, None, None, None) == -1
    at = lambda scale=0.0, flags=1, bb=b: L.kv_cache16_attend(  # noqa: E731
        c._h, ref(y), ref(bb), ref(r), ref(r), None, scale, 0, flags, None, 0, None)
    assert at(scale=-1.0) == -1 and at(scale=math.inf) == -1 and at(scale=math.nan) == -1 and at(flags=2) == -1
    empty = _batch(n_seqs=0, n_new=0)
    assert at(bb=empty) == 0                        # no rows: nothing to do, no pointer is looked at
    assert L.kv_cache16_append(c._h, ref(y), ref(empty), ref(r), ref(r), None, None, None, None) == 0
    for over, code in ((dict(lens=0), -1), (dict(tables=0), -1), (dict(table_stride=79), -1), (dict(table_stride=-80), -1),
                       (dict(lens=66), -5), (dict(tables=66), -5), (dict(cu_new=66), -5), (dict(errors=66), -5)):
        bb = _batch(**{**dict(lens=64, tables=64), **over})
        assert at(bb=bb) == code, over
        assert L.kv_cache16_append(c._h, ref(y), ref(bb), ref(r), ref(r), None, None, None, None) == code, over
    # the 8-bit cache's: queries want a rotation
    c8 = cache8.Cache8(**_kw())
    y8 = cache8._Layer(0, 0, 0, 0)
    assert cache8.lib().kv_cache8_append(c8._h, ref(y8), ref(b), ref(r), ref(r), None, ref(r), ref(r), None) == -1
    assert cache8.lib().kv_cache8_append(None, ref(y8), ref(b), ref(r), ref(r), None, None, None, None) == -1


class _Tensor:
    """Stands in for a CUDA tensor of some device where there is none: no byte of it is ever touched."""
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        t = torch.empty(*shape, dtype=dtype)
        self.device_index, self.dtype, self.shape, self.t = device, dtype, t.shape, t
        self.nbytes = t.nbytes
        for name in ("stride", "dim", "numel", "is_contiguous", "storage_offset", "untyped_storage"):
            setattr(self, name, getattr(t, name))

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 4096


def _on(device, **other):
    """The calls of a step of two sequences on one device, the arguments named by `other` on another."""
    at = lambda name, dtype, *shape: _Tensor(other.get(name, device), dtype, *shape)  # noqa: E731
    cache, eight = cache16.Cache16(**_kw()), cache8.Cache8(**_kw())
    layer = cache16.Layer(*(at(r, torch.bfloat16, 64 * 16 * 8 * 128) for r in ("k", "v")))
    layer8 = cache8.Layer(*(at(r, torch.uint8, 64 * 16 * 8 * 128) for r in ("k", "v")),
                          *(at(r, torch.float32, 64, 8) for r in ("k", "v")))
    batch = cache8.Batch(at("tables", torch.int32, 2, 4), at("lens", torch.int32, 2), at("cu", torch.int32, 3), n_new=2)
    kv, q, out = (at(r, torch.bfloat16, 2, h, 128) for r, h in (("new", 8), ("q", 32), ("out", 32)))
    turn = cache8.Rotation(at("cos", torch.float32, 50, 64), at("sin", torch.float32, 50, 64))
    lse, ws = at("lse", torch.float32, 2, 32), at("workspace", torch.uint8, 1 << 24)
    return {"append": lambda **kw: cache.append(layer, batch, kv, kv, rotation=turn, q=q, q_out=out, **kw),
            "append8": lambda **kw: eight.append(layer8, batch, kv, kv, rotation=turn, q=q, q_out=out, **kw),
            "attend": lambda **kw: cache.attend(layer, batch, q, out, lse=lse, workspace=ws, **kw)}


@pytest.mark.parametrize("name", ["v", "sin", "lens", "cu"])
def test_a_layer_a_rotation_and_a_batch_are_on_one_device(name):
    with pytest.raises(ValueError):
        _on(1, **{name: 0})


@pytest.mark.parametrize("call,names", [("append", ("new", "q", "out")), ("append8", ("new", "q", "out")),
                                        ("attend", ("q", "out", "lse", "workspace"))])
def test_a_call_is_on_one_device_which_is_the_current_one(monkeypatch, call, names):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    others = [{n: 0} for n in names] + [dict(k=0, v=0), dict(tables=0, lens=0, cu=0)]
    if call != "attend":
        others.append(dict(cos=0, sin=0))
    for other in others:
        with pytest.raises(ValueError):
            _on(1, **other)[call](stream=64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        _on(1)[call](stream=64)


def test_python_refusals_on_the_cpu():
    for f in (lambda: cache16.Layer(torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)),
              lambda: cache8.Rotation(torch.zeros(4, 16), torch.zeros(4, 16)),
              lambda: cache8.Rotation.of(32, 10, device="cpu")):
        with pytest.raises(ValueError):
            f()


# ---- the reference itself
def test_reference_rotation_is_a_complex_product():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(7, 3, 32, generator=g, dtype=torch.float64)
    c, s = R.tables(100, 16)
    pos = [0, 1, 5, 99, 40, 7, 98]
    w = torch.complex(c.double(), s.double())[pos][:, None]
    for neighbours in (False, True):
        y = R.turn(x, pos, c, s, neighbours)
        a, b = (x[..., 0:16:2], x[..., 1:16:2]) if neighbours else (x[..., :8], x[..., 8:16])
        z = torch.complex(a, b) * w
        u, v = (y[..., 0:16:2], y[..., 1:16:2]) if neighbours else (y[..., :8], y[..., 8:16])
        assert torch.allclose(u, z.real) and torch.allclose(v, z.imag) and torch.equal(y[..., 16:], x[..., 16:])
    assert torch.isnan(R.turn(x, [100] * 7, c, s, False)[..., :16]).all()


def test_reference_attention_against_a_plain_softmax():
    su = R.Setup(D=32, H=2, T=5, lens=[13, 0, 40], dtype="bf16", layout="packed", dev="cpu")
    su.fill()
    q = su.values(3, 4)
    out, lse, _, _ = su.attend(2, 40, q, window=7)
    (k, ok), (v, _) = su.tokens(0, 2, 40), su.tokens(1, 2, 40)
    assert bool(ok.all())
    for i in range(3):
        for h in range(4):
            a, b = 37 + i - 6, 38 + i
            z = (q[i, h].double() @ k[a:b, h // 2].T) / 32 ** 0.5
            assert torch.allclose(out[i, h], z.softmax(-1) @ v[a:b, h // 2])
            assert torch.allclose(lse[i, h], z.logsumexp(-1))
