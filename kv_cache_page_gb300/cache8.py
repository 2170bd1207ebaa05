"""The live 8-bit KV cache: ctypes binding of ``include/kv_cache8.h``.

K and V stay in 8 bits (E4M3 codes in pages, a power-of-two scale for each page
and head).  ``Cache8.write`` quantises new tokens into their pages,
``Cache8.attend`` reads the codes themselves, ``Cache8.read`` gives tokens back in
16 bits.  Every step runs in the CUDA kernels of ``libkvcodec.so``; this module
checks the tensors' types, shapes and devices (one, the current one) and passes pointers.
Calls enqueue on the given stream (default: torch's current stream), allocate nothing and can be
captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional, Sequence

import torch

from . import codec as _codec
from .codec import KvCodecError  # noqa: F401  (what the calls raise)

ABI_VERSION = 1
BAD_PAGE = 1
STALLED = 2
CAUSAL = 1
_MAX_WINDOW = 0xffffffff  # positions are below 2^31: all of any sequence
EXPORTS = ("kv_cache8_create", "kv_cache8_destroy", "kv_cache8_write", "kv_cache8_read", "kv_cache8_attend",
           "kv_cache8_attend_workspace", "kv_cache8_abi_version")
_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


class _Geometry(C.Structure):
    _fields_ = [("abi_version", C.c_uint32), ("struct_size", C.c_uint32), ("dtype", C.c_uint32),
                ("head_dim", C.c_uint32), ("num_kv_heads", C.c_uint32), ("num_q_heads", C.c_uint32),
                ("block_tokens", C.c_uint32), ("reserved", C.c_uint32), ("num_blocks", C.c_uint64),
                ("stride_block", C.c_int64), ("stride_token", C.c_int64), ("stride_head", C.c_int64)]


class _Layer(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p)]


class _Batch(C.Structure):
    _fields_ = [("struct_size", C.c_uint32), ("n_seqs", C.c_uint32), ("n_new", C.c_uint32),
                ("max_new", C.c_uint32), ("max_len", C.c_uint32), ("table_width", C.c_uint32),
                ("table_stride", C.c_int64), ("tables", C.c_void_p), ("lens", C.c_void_p),
                ("cu_new", C.c_void_p), ("errors", C.c_void_p)]


class _Rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride_row", C.c_int64), ("stride_head", C.c_int64)]


_LIB = None


def lib():
    global _LIB
    if _LIB is None:
        L = _codec.lib()
        vp, st = C.c_void_p, C.POINTER
        L.kv_cache8_create.argtypes = [st(_Geometry), st(vp)]
        L.kv_cache8_destroy.argtypes = [vp]
        L.kv_cache8_write.argtypes = [vp, vp, vp, vp, vp, vp]
        L.kv_cache8_read.argtypes = [vp, vp, vp, vp, vp, vp]
        L.kv_cache8_attend.argtypes = [vp, vp, vp, vp, vp, vp, C.c_float, C.c_uint32, C.c_uint32, vp, C.c_uint64, vp]
        L.kv_cache8_attend_workspace.argtypes = [vp, vp, st(C.c_uint64)]
        L.kv_cache8_abi_version.restype = C.c_uint32
        for f in EXPORTS[:-1]:
            getattr(L, f).restype = C.c_int
        _LIB = L
    return _LIB


def _stream(stream, device):
    """The raw stream: torch's current one by its handle (a Stream object per call costs 3 us)."""
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(device) if raw else torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _one_device(tensors, what):
    """The device index that the tensors share."""
    device = tensors[0].get_device()
    if any(t.get_device() != device for t in tensors):
        raise ValueError(f"the tensors of a {what} must be on one device")
    return device


def _int32(t, name, n=None):
    if t.dtype != torch.int32 or not t.is_cuda:
        raise ValueError(f"{name} must be an int32 CUDA tensor")
    if n is not None and (t.dim() != 1 or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous, of {n} entries")
    return t.data_ptr()


class Layer:
    """K and V codes (uint8 CUDA tensors of the registered page layout) and their
    scales (float32 [num_blocks, num_kv_heads]) of one model layer."""

    def __init__(self, k, v, k_scale, v_scale):
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_cuda:
                raise ValueError(f"{name} must be a uint8 or float8_e4m3fn CUDA tensor")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = _one_device((k, v, k_scale, v_scale), "layer")
        self.code_bytes = min(t.untyped_storage().nbytes() - t.storage_offset() for t in (k, v))
        self.scales = min(k_scale.numel(), v_scale.numel())
        self._c = _Layer(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = C.addressof(self._c)


class Batch:
    """The sequences of a step, for every layer's calls.

    tables [n_seqs, width]: page of each run of block_tokens positions; lens
    [n_seqs]: tokens held, the new ones among them; cu_new [n_seqs + 1]: running
    sums of the new tokens, ``None`` for one each; n_new: their total.  max_new and
    max_len (0: not known) only choose how work is split.  errors [n_seqs] (int32,
    zeroed by the caller): BAD_PAGE is or-ed in where a token's page is none, STALLED where
    attention gave up a wait and left the sequence's output unspecified (without errors
    neither is told).  All are int32 CUDA tensors, read on the device when a call runs."""

    def __init__(self, tables, lens, cu_new=None, *, n_new: Optional[int] = None, max_new: int = 0,
                 max_len: int = 0, errors=None):
        n = lens.numel()
        if tables.dim() != 2 or tables.shape[0] != n or (tables.shape[1] > 1 and tables.stride(1) != 1):
            raise ValueError("tables must be [n_seqs, width] with entries side by side")
        if cu_new is None:
            n_new = n if n_new is None else n_new
        elif n_new is None:
            raise ValueError("n_new (the rows of the 16-bit tensors) is required with cu_new")
        self.tables, self.lens, self.cu_new, self.errors = tables, lens, cu_new, errors
        self.n_new = n_new
        self._c = _Batch(C.sizeof(_Batch), n, n_new, max_new, max_len, tables.shape[1], tables.stride(0),
                         _int32(tables, "tables"), _int32(lens, "lens", n),
                         None if cu_new is None else _int32(cu_new, "cu_new", n + 1),
                         None if errors is None else _int32(errors, "errors", n))
        self._ref = C.addressof(self._c)
        self.device = _one_device([t for t in (tables, lens, cu_new, errors) if t is not None], "batch")


class Cache8:
    """A registered cache geometry (one ``kv_cache8_t`` handle).  strides: (block,
    token, head) in codes of the page layout; default [block, token, head, D]."""

    def __init__(self, *, dtype: str, head_dim: int, num_kv_heads: int, num_q_heads: int, block_tokens: int,
                 num_blocks: int, strides: Optional[Sequence[int]] = None, geometry_overrides=None):
        if strides is None:
            strides = (block_tokens * num_kv_heads * head_dim, num_kv_heads * head_dim, head_dim)
        g = _Geometry(ABI_VERSION, C.sizeof(_Geometry), _codec.DT[dtype], head_dim, num_kv_heads, num_q_heads,
                      block_tokens, 0, num_blocks, *strides)
        for k, v in (geometry_overrides or {}).items():
            setattr(g, k, v)
        self.dtype = _DTYPES[dtype]
        self.head_dim, self.num_kv_heads, self.num_q_heads = head_dim, num_kv_heads, num_q_heads
        self.block_tokens, self.num_blocks, self.strides = block_tokens, num_blocks, tuple(strides)
        # bytes a layer's code tensors and entries its scale tensors have at least
        self._codes = (strides[0] * (num_blocks - 1) + strides[1] * (block_tokens - 1) +
                       strides[2] * (num_kv_heads - 1) + head_dim)
        self._scales = num_blocks * num_kv_heads
        L = lib()
        self._write, self._read, self._attend = L.kv_cache8_write, L.kv_cache8_read, L.kv_cache8_attend
        h = C.c_void_p()
        self._h = None
        _codec._check(lib().kv_cache8_create(C.byref(g), C.byref(h)), "kv_cache8_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().kv_cache8_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def new_layer(self, device="cuda") -> Layer:
        """A zeroed layer of the registered geometry."""
        codes = [torch.zeros(self._codes, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(self.num_blocks, self.num_kv_heads, device=device) for _ in range(2)]
        return Layer(*codes, *scales)

    def _layer(self, layer, batch):
        if layer.code_bytes < self._codes or layer.scales < self._scales:
            raise ValueError("the layer's tensors are smaller than the registered geometry")
        if layer.device != batch.device or torch.cuda.current_device() != batch.device:
            raise ValueError("the layer and the batch must be on the current CUDA device")
        return layer._ref

    def _rows(self, t, batch, heads, name):
        if t.dtype is not self.dtype or not t.is_cuda or t.get_device() != batch.device:
            raise ValueError(f"{name} must be a {self.dtype} CUDA tensor on the batch's device")
        row, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
        if one != 1 or t.shape != (batch.n_new, heads, self.head_dim):
            raise ValueError(f"{name} must be [{batch.n_new}, {heads}, {self.head_dim}] with values side by side")
        return _Rows(t.data_ptr(), row, head)

    def write(self, layer: Layer, batch: Batch, k, v, stream=None):
        """Quantise the batch's new tokens (k, v: [n_new, num_kv_heads, head_dim]) into
        their pages; a page's scale grows where the new values need it, and its earlier
        codes are rewritten under the grown scale."""
        kr, vr = self._rows(k, batch, self.num_kv_heads, "k"), self._rows(v, batch, self.num_kv_heads, "v")
        rc = self._write(self._h, self._layer(layer, batch), batch._ref, C.addressof(kr), C.addressof(vr),
                         _stream(stream, batch.device))
        if rc:
            _codec._check(rc, "kv_cache8_write")

    def read(self, layer: Layer, batch: Batch, k, v, stream=None):
        """The batch's new tokens back in 16 bits, into k and v."""
        kr, vr = self._rows(k, batch, self.num_kv_heads, "k"), self._rows(v, batch, self.num_kv_heads, "v")
        rc = self._read(self._h, self._layer(layer, batch), batch._ref, C.addressof(kr), C.addressof(vr),
                        _stream(stream, batch.device))
        if rc:
            _codec._check(rc, "kv_cache8_read")

    def attend_workspace(self, batch: Batch) -> int:
        """Bytes of the workspace that ``attend`` wants for this batch's sizes."""
        n = C.c_uint64()
        _codec._check(lib().kv_cache8_attend_workspace(self._h, batch._ref, C.byref(n)), "kv_cache8_attend_workspace")
        return n.value

    def attend(self, layer: Layer, batch: Batch, q, out, *, lse=None, scale: Optional[float] = None,
               causal: bool = True, window: int = 0, workspace=None, stream=None):
        """Attention of the new tokens' queries (q, out: [n_new, num_q_heads, head_dim])
        over their sequences; lse (float32 [n_new, num_q_heads]): the scores' log-sum-exp.
        A row that sees no key gets out = 0, lse = -inf.  workspace: a CUDA tensor of at
        least ``attend_workspace(batch)`` bytes, zero-filled before its first use, then good
        for any batch or cache, not shared by calls that may run at the same time."""
        qr, outr = self._rows(q, batch, self.num_q_heads, "q"), self._rows(out, batch, self.num_q_heads, "out")
        at = None
        if lse is not None:
            if lse.dtype is not torch.float32 or not lse.is_cuda or lse.shape != (batch.n_new, self.num_q_heads) or \
                    not lse.is_contiguous() or lse.get_device() != batch.device:
                raise ValueError(f"lse must be a contiguous float32 CUDA tensor [{batch.n_new}, {self.num_q_heads}] on "
                                 "the batch's device")
            at = lse.data_ptr()
        if scale is None:
            scale = 0.0
        elif not (scale > 0 and math.isfinite(C.c_float(scale).value) and C.c_float(scale).value > 0):
            raise ValueError("scale must be finite and positive in float32")  # (0 would stand for the default)
        if window < 0:
            raise ValueError("window must not be negative")
        window = min(window, _MAX_WINDOW)
        ws, nb = None, 0
        if workspace is not None:
            if not workspace.is_cuda or not workspace.is_contiguous() or workspace.get_device() != batch.device:
                raise ValueError("workspace must be a contiguous CUDA tensor on the batch's device")
            ws, nb = workspace.data_ptr(), workspace.nbytes
        rc = self._attend(self._h, self._layer(layer, batch), batch._ref, C.addressof(qr), C.addressof(outr), at, scale,
                          window, CAUSAL if causal else 0, ws, nb, _stream(stream, batch.device))
        if rc:
            _codec._check(rc, "kv_cache8_attend")
