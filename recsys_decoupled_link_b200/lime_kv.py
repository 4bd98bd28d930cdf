"""Thin Python binding of the paged 8-bit history cache (include/lime_kv.h).

Like ``lime``, the functions keep the C names and only marshal arguments:
torch tensors are passed as raw device pointers, the stream is torch's current
stream unless one is given, and every numeric step runs in the library's
kernels.  ``HistoryCache`` owns the pool, the block table and the free stack
of a serving program and chains the calls.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from .lime import (LIME_BF16, LIME_ERR_SHAPE, LIME_F32, LimeError, _check, _lib, _ptr, _stream,
                   lime_get_status, lime_workspace_init)

LIME_FLAG_BAD_BLOCK, LIME_FLAG_NO_BLOCKS, LIME_FLAG_NONFINITE = 8, 16, 32


class lime_kv_dims(ctypes.Structure):
    _fields_ = [("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("dh", ctypes.c_int32),
                ("block", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("n_blocks", ctypes.c_int64)]


def _sign():
    P, I64, SZ, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    D = ctypes.POINTER(lime_kv_dims)
    sig = {
        "lime_kv_workspace_bytes": (SZ, [D, I64, I64]),
        "lime_kv_reserve": (I32, [D, I64, P, P, I64, P, P, I64, P, P, P, P, P, SZ, P]),
        "lime_kv_release": (I32, [D, I64, P, P, P, P, I64, P, P, P, P, SZ, P]),
        "lime_kv_append": (I32, [D, P, I64, P, I64, I64, P, P, P, P, P, SZ, P]),
        "lime_kv_attention": (I32, [D, I64, P, I64, P, I64, P, P, P, P, P, ctypes.c_float, I32,
                                    P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = res, args


_sign()
EXPORTED = ("lime_kv_workspace_bytes", "lime_kv_reserve", "lime_kv_release", "lime_kv_append",
            "lime_kv_attention")


def make_kv_dims(Hq: int, Hkv: int, dh: int, block: int, n_blocks: int, max_blocks: int,
                 dtype) -> lime_kv_dims:
    dt = LIME_BF16 if dtype in (torch.bfloat16, "bf16", LIME_BF16) else LIME_F32
    return lime_kv_dims(Hq, Hkv, dh, block, max_blocks, dt, n_blocks)


def lime_kv_workspace_bytes(dims: lime_kv_dims, B: int, total_q: int) -> int:
    return int(_lib.lime_kv_workspace_bytes(ctypes.byref(dims), B, total_q))


class KvWorkspace:
    """A device workspace sized by lime_kv_workspace_bytes and initialised."""

    def __init__(self, dims: lime_kv_dims, B: int, total_q: int, device="cuda", stream=None):
        n = lime_kv_workspace_bytes(dims, B, total_q)
        if n == 0:
            raise LimeError("lime_kv_workspace_bytes", LIME_ERR_SHAPE)
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)
        self.nbytes = n
        lime_workspace_init(self, stream=stream)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())


def _device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() else 0


def _want(name: str, t: torch.Tensor, dtype, shape):
    """A tensor's type, device and shape (-1: any size), checked before its pointer is passed."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.get_device() != _device():
        raise ValueError(f"{name}: liblime takes tensors of the current device")
    if t.dim() != len(shape) or any(w not in (-1, g) for w, g in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")


def _rows(name: str, t: torch.Tensor, dims: lime_kv_dims, heads: int):
    """Pointer and row pitch of packed rows [n, heads, dh]; rows may be strided."""
    _want(name, t, torch.bfloat16 if dims.dtype == LIME_BF16 else torch.float32,
          (-1, heads, dims.dh))
    if (heads > 1 and t.stride(1) != dims.dh) or t.stride(2) != 1:
        raise ValueError(f"{name}: the heads of a row have to be contiguous")
    ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), heads * dims.dh)
    return ctypes.c_void_p(t.data_ptr()), ld


def _pool(dims: lime_kv_dims, k_cache, v_cache, scale):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _want(name, t, torch.int8, (dims.n_blocks, dims.Hkv, dims.block, dims.dh))
    _want("scale", scale, torch.float32, (dims.n_blocks, dims.Hkv, 2))


def lime_kv_reserve(dims, lens, new_offsets, block_table, free_blocks, n_free, lens_out,
                    n_free_out, slot_map, ws: KvWorkspace, stream=None):
    B = lens.shape[0]
    for name, t, dtype, shape in (
            ("lens", lens, torch.int32, (B,)), ("new_offsets", new_offsets, torch.int64, (B + 1,)),
            ("block_table", block_table, torch.int32, (B, dims.max_blocks)),
            ("free_blocks", free_blocks, torch.int32, (-1,)),
            ("n_free", n_free, torch.int32, (1,)), ("lens_out", lens_out, torch.int32, (B,)),
            ("n_free_out", n_free_out, torch.int32, (1,)),
            ("slot_map", slot_map, torch.int64, (-1,))):
        _want(name, t, dtype, shape)
    _check("lime_kv_reserve", _lib.lime_kv_reserve(
        ctypes.byref(dims), B, _ptr(lens), _ptr(new_offsets), slot_map.shape[0],
        _ptr(block_table), _ptr(free_blocks), free_blocks.shape[0], _ptr(n_free), _ptr(lens_out),
        _ptr(n_free_out), _ptr(slot_map), ws.ptr, ws.nbytes, _stream(stream)))


def lime_kv_release(dims, lens, keep: Optional[torch.Tensor], block_table, free_blocks, n_free,
                    lens_out, n_free_out, ws: KvWorkspace, stream=None):
    B = lens.shape[0]
    for name, t, dtype, shape in (
            ("lens", lens, torch.int32, (B,)),
            ("block_table", block_table, torch.int32, (B, dims.max_blocks)),
            ("free_blocks", free_blocks, torch.int32, (-1,)),
            ("n_free", n_free, torch.int32, (1,)), ("lens_out", lens_out, torch.int32, (B,)),
            ("n_free_out", n_free_out, torch.int32, (1,))):
        _want(name, t, dtype, shape)
    if keep is not None:
        _want("keep", keep, torch.int32, (B,))
    _check("lime_kv_release", _lib.lime_kv_release(
        ctypes.byref(dims), B, _ptr(lens), _ptr(keep), _ptr(block_table), _ptr(free_blocks),
        free_blocks.shape[0], _ptr(n_free), _ptr(lens_out), _ptr(n_free_out), ws.ptr, ws.nbytes,
        _stream(stream)))


def lime_kv_append(dims, K, V, slot_map, k_cache, v_cache, scale, ws: KvWorkspace, stream=None):
    """K, V [n, Hkv, dh] with any row pitch; slot_map int64 [n]."""
    k, ldk = _rows("K", K, dims, dims.Hkv)
    v, ldv = _rows("V", V, dims, dims.Hkv)
    _want("slot_map", slot_map, torch.int64, (K.shape[0],))
    _want("V", V, K.dtype, K.shape)
    _pool(dims, k_cache, v_cache, scale)
    _check("lime_kv_append", _lib.lime_kv_append(
        ctypes.byref(dims), k, ldk, v, ldv, K.shape[0], _ptr(slot_map), _ptr(k_cache),
        _ptr(v_cache), _ptr(scale), ws.ptr, ws.nbytes, _stream(stream)))


def lime_kv_attention(dims, Q, q_offsets, block_table, lens, k_cache, v_cache, scale, O, lse,
                      ws: KvWorkspace, sm_scale: Optional[float] = None, causal: bool = False,
                      stream=None):
    """Q [n, Hq, dh] with any row pitch; lse fp32 [n, Hq] or None; sm_scale 1/sqrt(dh) if None."""
    B = lens.shape[0]
    q, ldq = _rows("Q", Q, dims, dims.Hq)
    _want("q_offsets", q_offsets, torch.int64, (B + 1,))
    _want("block_table", block_table, torch.int32, (B, dims.max_blocks))
    _want("lens", lens, torch.int32, (B,))
    _want("O", O, Q.dtype, Q.shape)
    if lse is not None:
        _want("lse", lse, torch.float32, Q.shape[:2])
    _pool(dims, k_cache, v_cache, scale)
    sm = 1.0 / math.sqrt(dims.dh) if sm_scale is None else sm_scale
    _check("lime_kv_attention", _lib.lime_kv_attention(
        ctypes.byref(dims), B, q, ldq, _ptr(q_offsets), Q.shape[0], _ptr(block_table), _ptr(lens),
        _ptr(k_cache), _ptr(v_cache), _ptr(scale), sm, int(causal), _ptr(O), _ptr(lse), ws.ptr,
        ws.nbytes, _stream(stream)))


class HistoryCache:
    """The cache of a serving program with B request rows: pool, block table, free stack.

    ``append`` finds room for new rows and writes them, ``attend`` lets query
    rows attend over everything cached, ``release`` shortens requests.  Calls
    are asynchronous on the current stream and belong on one stream.  The
    lengths and the stack's height alternate between two buffers, since the
    library's calls read one and write the other; ``append`` and ``release``
    advance that state on the host, so inside a captured graph use the calls
    themselves."""

    def __init__(self, dims: lime_kv_dims, B: int, max_q: int = 0, device="cuda"):
        self.dims, self.B = dims, B
        new = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device=device)
        shape = (dims.n_blocks, dims.Hkv, dims.block, dims.dh)
        self.k, self.v = (torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2))
        self.scale = torch.empty(dims.n_blocks, dims.Hkv, 2, device=device)
        self.table = new(B, dims.max_blocks) - 1
        self.free = torch.arange(dims.n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self.lens, self._lens = new(B), new(B)
        self.n_free, self._n_free = new(1) + dims.n_blocks, new(1)
        self.ws = KvWorkspace(dims, B, max_q, device=device)
        self.max_q = max_q

    def _advance(self):
        self.lens, self._lens = self._lens, self.lens
        self.n_free, self._n_free = self._n_free, self.n_free

    def append(self, K: torch.Tensor, V: torch.Tensor, new_offsets: torch.Tensor) -> torch.Tensor:
        """Caches K, V [n, Hkv, dh], request u's rows at [new_offsets[u], new_offsets[u+1]);
        returns the slots (-1: no room)."""
        slots = torch.empty(K.shape[0], dtype=torch.int64, device=K.device)
        lime_kv_reserve(self.dims, self.lens, new_offsets, self.table, self.free, self.n_free,
                        self._lens, self._n_free, slots, self.ws)
        self._advance()
        lime_kv_append(self.dims, K, V, slots, self.k, self.v, self.scale, self.ws)
        return slots

    def attend(self, Q: torch.Tensor, q_offsets: torch.Tensor, causal: bool = False,
               sm_scale: Optional[float] = None, lse: Optional[torch.Tensor] = None):
        """Attention of Q [n, Hq, dh] over the cached rows; returns O [n, Hq, dh]."""
        if Q.shape[0] > self.max_q:
            self.ws = KvWorkspace(self.dims, self.B, Q.shape[0], device=Q.device)
            self.max_q = Q.shape[0]
        O = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device)
        lime_kv_attention(self.dims, Q, q_offsets, self.table, self.lens, self.k, self.v,
                          self.scale, O, lse, self.ws, sm_scale, causal)
        return O

    def release(self, keep: Optional[torch.Tensor] = None):
        """Keeps the first keep[u] rows of every request (None: nothing)."""
        lime_kv_release(self.dims, self.lens, keep, self.table, self.free, self.n_free,
                        self._lens, self._n_free, self.ws)
        self._advance()

    def status(self, stream=None) -> int:
        return lime_get_status(self.ws, stream)
