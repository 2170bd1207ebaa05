"""The live 16-bit KV cache: ctypes binding of ``include/kv_cache16.h``.

K and V stay in the engine's FP16/BF16 pages, the layouts that the page codec encodes
and restores.  ``Cache16.append`` puts new tokens into their pages, the keys turned by
their positions on the way, and turns the same tokens' queries; ``Cache16.attend``
reads the pages.  Batches and rotations are those of the 8-bit cache
(``cache8.Batch``, ``cache8.Rotation``), so one batch serves layers of both kinds.
Every step runs in the CUDA kernels of ``libkvcodec.so``; this module checks the tensors'
types, shapes and devices (one, the current one) and passes pointers.  Calls enqueue
on the given stream (default: torch's current stream), allocate nothing and can be
captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

import torch

from . import cache8 as _cache8
from . import codec as _codec
from .cache8 import BAD_PAGE, BAD_POSITION, Batch, KvCodecError, Rotation  # noqa: F401

ABI_VERSION = 1
EXPORTS = ("kv_cache16_create", "kv_cache16_destroy", "kv_cache16_append", "kv_cache16_attend",
           "kv_cache16_attend_workspace", "kv_cache16_abi_version")


class _Layer(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p)]


_LIB = None


def lib():
    global _LIB
    if _LIB is None:
        L = _codec.lib()
        vp, st = C.c_void_p, C.POINTER
        L.kv_cache16_create.argtypes = [st(_cache8._Geometry), st(vp)]
        L.kv_cache16_destroy.argtypes = [vp]
        L.kv_cache16_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.kv_cache16_attend.argtypes = [vp, vp, vp, vp, vp, vp, C.c_float, C.c_uint32, C.c_uint32, vp, C.c_uint64, vp]
        L.kv_cache16_attend_workspace.argtypes = [vp, vp, st(C.c_uint64)]
        L.kv_cache16_abi_version.restype = C.c_uint32
        for f in EXPORTS[:-1]:
            getattr(L, f).restype = C.c_int
        _LIB = L
    return _LIB


class Layer:
    """K and V pages of one model layer (float16 or bfloat16 CUDA tensors of the registered page layout; of a
    packed tensor [block, head, token, 2 D]: its views ``[..., :D]`` and ``[..., D:]``)."""

    def __init__(self, k, v):
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.float16, torch.bfloat16) or t.dtype != k.dtype or not t.is_cuda:
                raise ValueError(f"{name} must be a float16 or bfloat16 CUDA tensor, k and v of one type")
        self.k, self.v, self.dtype = k, v, k.dtype
        self.device = _cache8._one_device((k, v), "layer")
        self.values = min(t.untyped_storage().nbytes() // 2 - t.storage_offset() for t in (k, v))
        self._c = _Layer(k.data_ptr(), v.data_ptr())
        self._ref = C.addressof(self._c)


class Cache16(_cache8._Cache):
    """A registered cache geometry (one ``kv_cache16_t`` handle).  strides: (block,
    token, head) in values of the page layout; default [block, token, head, D]."""

    def __init__(self, *, dtype: str, head_dim: int, num_kv_heads: int, num_q_heads: int, block_tokens: int,
                 num_blocks: int, strides: Optional[Sequence[int]] = None, geometry_overrides=None):
        if strides is None:
            strides = (block_tokens * num_kv_heads * head_dim, num_kv_heads * head_dim, head_dim)
        g = _cache8._Geometry(ABI_VERSION, C.sizeof(_cache8._Geometry), _codec.DT[dtype], head_dim, num_kv_heads,
                              num_q_heads, block_tokens, 0, num_blocks, *strides)
        for k, v in (geometry_overrides or {}).items():
            setattr(g, k, v)
        self.dtype = _cache8._DTYPES[dtype]
        self.head_dim, self.num_kv_heads, self.num_q_heads = head_dim, num_kv_heads, num_q_heads
        self.block_tokens, self.num_blocks, self.strides = block_tokens, num_blocks, tuple(strides)
        # values a layer's tensors have at least, from their first one
        self._values = (strides[0] * (num_blocks - 1) + strides[1] * (block_tokens - 1) +
                        strides[2] * (num_kv_heads - 1) + head_dim)
        L = lib()
        self._append, self._attend = L.kv_cache16_append, L.kv_cache16_attend
        h = C.c_void_p()
        self._h = None
        _codec._check(L.kv_cache16_create(C.byref(g), C.byref(h)), "kv_cache16_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().kv_cache16_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def new_layer(self, device="cuda") -> Layer:
        """A zeroed layer of the registered geometry, K and V apart."""
        return Layer(*(torch.zeros(self._values, dtype=self.dtype, device=device) for _ in range(2)))

    def _layer(self, layer, batch):
        if layer.dtype is not self.dtype or layer.values < self._values:
            raise ValueError("the layer's tensors are smaller than the registered geometry, or of another type")
        if layer.device != batch.device or torch.cuda.current_device() != batch.device:
            raise ValueError("the layer and the batch must be on the current CUDA device")
        return layer._ref

    def append(self, layer: Layer, batch: Batch, k, v, *, rotation: Optional[Rotation], q=None, q_out=None, stream=None):
        """The batch's new tokens (k, v: [n_new, num_kv_heads, head_dim]) into their pages, the keys turned by their
        positions (rotation None: as they are).  q, q_out ([n_new, num_q_heads, head_dim], both or neither): the tokens'
        queries, turned; q_out may be q itself.  Rows without a position get q_out = 0; those past the rotation's table
        get NaN in the turned channels of keys and queries, and BAD_POSITION; a token without a page is not written, and BAD_PAGE."""
        self._append_call(self._append, "kv_cache16_append", layer, batch, k, v, rotation, q, q_out, stream)

    def attend_workspace(self, batch: Batch) -> int:
        """Bytes of the workspace that ``attend`` wants: the same for every batch that has new tokens."""
        n = C.c_uint64()
        _codec._check(lib().kv_cache16_attend_workspace(self._h, batch._ref, C.byref(n)), "kv_cache16_attend_workspace")
        return n.value

    def attend(self, layer: Layer, batch: Batch, q, out, *, lse=None, scale: Optional[float] = None,
               causal: bool = True, window: int = 0, workspace=None, stream=None):
        """Attention of the new tokens' queries (q, out: [n_new, num_q_heads, head_dim])
        over their sequences; lse (float32 [n_new, num_q_heads]): the scores' log-sum-exp.
        A row that sees no key gets out = 0, lse = -inf.  Made for one or a few new tokens a sequence.
        workspace: a CUDA tensor of at least ``attend_workspace(batch)`` bytes, zero-filled before its
        first use, then good for any batch or cache (8-bit ones too), not shared by calls that may
        run at the same time."""
        self._attend_call(self._attend, "kv_cache16_attend", layer, batch, q, out, lse, scale, causal, window, workspace,
                          stream)
