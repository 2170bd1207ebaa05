"""Host-only checks of the live 8-bit cache (no GPU): exports, structures,
refusals, workspace sizes; and the 64-bit reference that the GPU tests use."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import cache8_ref as R
from kv_cache_page_gb300 import build as kbuild
from kv_cache_page_gb300 import cache8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "kv_cache8.h")).read()
    names = set(re.findall(r"^\s*\w+\s+(kv_cache8_\w+)\s*\(", text, re.M))
    assert names == set(cache8.EXPORTS)
    for lib in (cache8.lib(), C.CDLL(kbuild.build(debug=True))):
        for n in names:
            assert hasattr(lib, n), n
    assert cache8.lib().kv_cache8_abi_version() == cache8.ABI_VERSION


def test_the_binding_names_every_error_bit():
    text = open(os.path.join(ROOT, "include", "kv_cache8.h")).read()
    bits = {n: int(v) for n, v in re.findall(r"^#define KV_CACHE8_(BAD_PAGE|STALLED|CAUSAL) (\d+)u", text, re.M)}
    assert bits == {"BAD_PAGE": cache8.BAD_PAGE, "STALLED": cache8.STALLED, "CAUSAL": cache8.CAUSAL}


def test_structure_sizes():
    assert [C.sizeof(x) for x in (cache8._Geometry, cache8._Layer, cache8._Batch, cache8._Rows)] == [64, 32, 64, 24]


def _kw(**over):
    kw = dict(dtype="bf16", head_dim=128, num_kv_heads=8, num_q_heads=32, block_tokens=16, num_blocks=64)
    kw.update(over)
    return kw


@pytest.mark.parametrize("over,code", [
    (dict(head_dim=96), -2),
    (dict(head_dim=512), -2),
    (dict(num_kv_heads=0), -1),
    (dict(num_q_heads=12), -1),                 # not a multiple of 8
    (dict(num_q_heads=0), -1),
    (dict(num_q_heads=8 * 65), -1),
    (dict(block_tokens=0), -1),
    (dict(block_tokens=32769), -1),
    (dict(num_blocks=0), -1),
    (dict(num_blocks=1 << 31), -1),
    (dict(geometry_overrides={"dtype": 3}), -1),
    (dict(geometry_overrides={"reserved": 1}), -1),
    (dict(geometry_overrides={"abi_version": 2}), -7),
    (dict(geometry_overrides={"struct_size": 56}), -7),
    (dict(strides=(16 * 8 * 128, 8 * 128, 120)), -5),
    (dict(strides=(16 * 8 * 128, 8 * 128, 64)), -3),     # heads overlap
    (dict(strides=(8 * 128, 8 * 128, 128)), -3),         # pages overlap
    (dict(strides=(16 * 8 * 128, 0, 128)), -3),
])
def test_geometry_refusals(over, code):
    with pytest.raises(cache8.KvCodecError) as e:
        cache8.Cache8(**_kw(**over))
    assert e.value.code == code


def test_accepted_layouts():
    cache8.Cache8(**_kw()).close()
    cache8.Cache8(**_kw(strides=(16 * 8 * 128, 128, 16 * 128))).close()        # pages by head
    cache8.Cache8(**_kw(strides=(2 * 16 * 8 * 128, 8 * 128, 128))).close()     # K and V pages interleaved
    cache8.Cache8(**_kw(num_blocks=1, num_kv_heads=1, num_q_heads=5, strides=(16, 128, 16))).close()
    cache8.Cache8(**_kw(block_tokens=1, strides=(1024, 1024, 128))).close()


def _batch(**over):
    b = dict(struct_size=64, n_seqs=4, n_new=4, max_new=1, max_len=1000, table_width=80, table_stride=80)
    b.update(over)
    return cache8._Batch(**b)


def _workspace(cache, b):
    n = C.c_uint64()
    return cache8.lib().kv_cache8_attend_workspace(cache._h, C.byref(b), C.byref(n)), n.value


@pytest.mark.parametrize("over,code", [
    (dict(struct_size=56), -7),
    (dict(n_seqs=65536, n_new=65536), -1),
    (dict(n_new=5), -1),                           # one new token each without cu_new
    (dict(n_seqs=0, n_new=3, cu_new=64), -1),
    (dict(n_new=1 << 30, cu_new=64), -1),          # rows past 31 bits
])
def test_batch_refusals(over, code):
    c = cache8.Cache8(**_kw())
    assert _workspace(c, _batch(**over))[0] == code


def test_workspace_sizes():
    c = cache8.Cache8(**_kw())
    rc, few = _workspace(c, _batch(n_seqs=1, n_new=1, max_len=100000, table_width=10000, table_stride=10000))
    assert rc == 0 and few > 0                      # one long sequence: split into ranges
    assert _workspace(c, _batch(n_seqs=1, n_new=1, max_len=50))[1] == 0   # one range
    assert _workspace(c, _batch(n_seqs=0, n_new=0)) == (0, 0)
    # a bound that is not given is the tables' reach
    assert _workspace(c, _batch(max_len=0))[1] == _workspace(c, _batch(max_len=80 * 16))[1]


def test_workspace_tickets_take_the_same_place_for_every_batch():
    """What is left of a workspace's bytes once the partial results are taken off does not depend on the batch."""
    left = set()
    for D, H, HQ in ((128, 8, 32), (64, 1, 7), (256, 4, 4), (32, 2, 128)):
        c = cache8.Cache8(**_kw(head_dim=D, num_kv_heads=H, num_q_heads=HQ, num_blocks=1 << 20))
        for n in list(range(1, 130)) + [200, 400, 700]:
            for cu in (0, 64):
                for new in ((1,) if not cu else (1, 5, 300, 4000)):
                    b = _batch(n_seqs=n, n_new=n * new, max_new=new, max_len=65536, table_width=4096, table_stride=4096,
                               cu_new=cu)
                    rc, total = _workspace(c, b)
                    assert rc == 0
                    if total:
                        left.add(total % (16 * (D + 2) * 4) - 16384 % (16 * (D + 2) * 4))
    assert left == {0}


def test_null_arguments():
    L, n = cache8.lib(), C.c_uint64()
    c = cache8.Cache8(**_kw())
    b, y = _batch(lens=64, tables=64), cache8._Layer(0, 0, 0, 0)
    r = cache8._Rows(0, 1024, 128)
    assert L.kv_cache8_create(None, C.byref(C.c_void_p())) == -1
    assert L.kv_cache8_destroy(None) == -1
    assert L.kv_cache8_attend_workspace(c._h, None, C.byref(n)) == -1
    assert L.kv_cache8_attend_workspace(c._h, C.addressof(b), None) == -1
    for f in (L.kv_cache8_write, L.kv_cache8_read):
        assert f(None, C.addressof(y), C.addressof(b), C.addressof(r), C.addressof(r), None) == -1
        assert f(c._h, C.addressof(y), None, C.addressof(r), C.addressof(r), None) == -1
    at = lambda scale=0.0, flags=1, bb=b: L.kv_cache8_attend(  # noqa: E731
        c._h, C.addressof(y), C.addressof(bb), C.addressof(r), C.addressof(r), None, scale, 0, flags, None, 0, None)
    assert at(scale=-1.0) == -1 and at(scale=math.inf) == -1 and at(scale=math.nan) == -1 and at(flags=2) == -1
    empty = _batch(n_seqs=0, n_new=0)
    assert at(bb=empty) == 0                        # no rows: nothing to do, no pointer is looked at
    # checked before any pointer is used on a device
    for over, code in ((dict(lens=0), -1), (dict(tables=0), -1), (dict(table_stride=79), -1), (dict(table_stride=-80), -1),
                       (dict(lens=66), -5), (dict(tables=66), -5), (dict(cu_new=66), -5), (dict(errors=66), -5)):
        bb = _batch(**{**dict(lens=64, tables=64), **over})
        assert at(bb=bb) == code, over


def test_python_refusals_on_the_cpu():
    c = cache8.Cache8(**_kw())
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        cache8.Batch(torch.zeros(2, 4, **i32), torch.zeros(2, **i32))              # not on a GPU
    with pytest.raises(ValueError):
        cache8.Layer(*[torch.zeros(4, dtype=torch.uint8)] * 2, *[torch.zeros(4)] * 2)
    with pytest.raises(ValueError):
        cache8.Batch(torch.zeros(3, 4, **i32), torch.zeros(2, **i32))
    with pytest.raises(ValueError):
        cache8.Batch(torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32))   # n_new missing
    c.close()


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
    """The arguments of a step of two sequences on one device, those named by `other` on another."""
    at = lambda name, dtype, *shape: _Tensor(other.get(name, device), dtype, *shape)  # noqa: E731
    cache = cache8.Cache8(**_kw())
    layer = cache8.Layer(*(at(r, torch.uint8, 64 * 16 * 8 * 128) for r in ("k", "v")),
                         *(at(r, torch.float32, 64, 8) for r in ("k_scale", "v_scale")))
    batch = cache8.Batch(at("tables", torch.int32, 2, 4), at("lens", torch.int32, 2), at("cu", torch.int32, 3), n_new=2,
                         errors=at("errors", torch.int32, 2))
    kv, q, out = (at(r, torch.bfloat16, 2, h, 128) for r, h in (("new", 8), ("q", 32), ("out", 32)))
    lse, ws = at("lse", torch.float32, 2, 32), at("workspace", torch.uint8, 1 << 24)
    return {"write": lambda **kw: cache.write(layer, batch, kv, kv, **kw),
            "read": lambda **kw: cache.read(layer, batch, kv, kv, **kw),
            "attend": lambda **kw: cache.attend(layer, batch, q, out, lse=lse, workspace=ws, **kw)}


@pytest.mark.parametrize("name", ["v", "k_scale", "v_scale", "lens", "cu", "errors"])
def test_a_layer_and_a_batch_are_on_one_device(name):
    with pytest.raises(ValueError):
        _on(1, **{name: 0})


@pytest.mark.parametrize("call,names", [("write", ("new",)), ("read", ("new",)), ("attend", ("q", "out", "lse", "workspace"))])
def test_a_call_is_on_one_device_which_is_the_current_one(monkeypatch, call, names):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for name in names:
        with pytest.raises(ValueError):
            _on(1, **{name: 0})[call](stream=64)
    for name in (dict(k=0, v=0, k_scale=0, v_scale=0), dict(tables=0, lens=0, cu=0, errors=0)):
        with pytest.raises(ValueError):
            _on(1, **name)[call](stream=64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        _on(1)[call](stream=64)


def test_a_stall_of_any_role_is_reported():
    """Every role of the prompt kernel may be the one whose wait runs out, the products' warp having finished: the report
    comes from the mark that they share, after the barrier that all of them reach."""
    text = open(os.path.join(ROOT, "kv_cache_page_gb300", "csrc", "cache8_prompt.cu")).read()
    kernel = text[text.index("c8_prompt_kernel(const __grid_constant__"):]
    report = [m.start() for m in re.finditer("KV_CACHE8_STALLED", kernel)]
    assert len(report) == 1 and report[0] > kernel.rindex("barrier.sync 0;")
    assert "if (tid == 0 && *stop)" in kernel


def test_the_write_kernel_reads_what_it_stores_with_ordinary_loads():
    """Pages and scales change in that kernel: the read-only path (ld.global.nc) promises nothing about them."""
    text = open(os.path.join(ROOT, "kv_cache_page_gb300", "csrc", "cache8_rw.cu")).read()
    kernel = text[text.index("c8_write_kernel(const __grid_constant__"):text.index("c8_read_kernel(const __grid_constant__")]
    read_only = re.findall(r"\b(ldg_\w+|ld_nc\w*|ld_stream\w*|__ldg)(?:<\w+>)?\(([^)]*)\)", kernel)
    assert read_only and all(at == "at" for _, at in read_only)      # the new values
    assert kernel.count("const uint16_t* at = src;") == 3
    assert "*at = c;" in kernel and "uint2 c = *at;" in kernel       # the codes held
    assert "ld_held_f32(scale_at)" in kernel


# ---- the reference itself, against torch's E4M3 conversions
def test_reference_codes_match_the_format():
    bits = torch.arange(256, dtype=torch.uint8)
    t = bits.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(t, nan=1e9), torch.nan_to_num(R.TABLE, nan=1e9))
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g) * torch.exp(3 * torch.randn(20000, generator=g))
    x = torch.cat([x.clamp(-448, 448), t[~torch.isnan(t)].float(), torch.tensor([0.0, -0.0, 2.0 ** -10, 2.0 ** -11])])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(R.encode(x.double()), want)
    assert R.encode(torch.tensor([math.inf, -math.inf, 500.0, math.nan], dtype=torch.float64)).tolist() == [126, 254, 126, 127]


def test_reference_exponent():
    for a, e in ((0.0, -60), (448.0, 0), (448.0001, 1), (224.0, -1), (1e-30, -60), (3e38, 119), (65504.0, 8)):
        assert R.page_exponent(a) == e


# ---- what a warpgroup has to do as one
def test_the_register_split_is_made_once_for_each_warpgroup():
    """setmaxnreg: all warps of a warpgroup execute the same instruction, so no two roles of one have calls of their own."""
    text = open(os.path.join(ROOT, "kv_cache_page_gb300", "csrc", "cache8_prompt.cu")).read()
    kernel = text[text.index("c8_prompt_kernel(const __grid_constant__"):]
    # one place for warps 0 .. 7, one for 8 .. 11 (before the branch that V's loaders begin), one for 12 .. 15
    assert kernel.count("regs_inc();") == 1 and kernel.count("regs_dec();") == 2
    assert re.search(r"if \(warp < kSoftWarps\) \{[^{}]*regs_inc\(\);", kernel)
    assert re.search(r"\} else if \(warp < kSoftWarps \+ kVWarps\) \{[^{}]*regs_dec\(\);[^{}]*\} else \{\s*regs_dec\(\);", kernel)
    # the split falls between warpgroups: warps 0 .. 7 take more, 8 .. 15 keep less, and the shares add up to the launch's
    warps = {n: int(v) for n, v in re.findall(r"(kSoftWarps|kVWarps|kKWarps) = (\d+)", text)}
    more, less = (int(re.search(r"setmaxnreg\.%s\.sync\.aligned\.u32 (\d+);" % d, text).group(1)) for d in ("inc", "dec"))
    soft, rest = warps["kSoftWarps"], warps["kVWarps"] + warps["kKWarps"] + 1
    assert soft % 4 == 0 and warps["kVWarps"] % 4 == 0 and rest % 4 == 0
    assert 32 * (soft * more + rest * less) <= 32 * (soft + rest) * 128
