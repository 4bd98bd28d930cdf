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

from .lime import LIME_BF16, LIME_ERR_SHAPE, LIME_F32, LimeError, _lib, lime_get_status

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
        "lime_kv_workspace_init": (I32, [P, SZ, P]),
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
EXPORTED = ("lime_kv_workspace_bytes", "lime_kv_workspace_init", "lime_kv_reserve",
            "lime_kv_release", "lime_kv_append", "lime_kv_attention")


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
        self.nbytes, self.address = n, self.buf.data_ptr()
        self.device = self.buf.get_device()
        lime_kv_workspace_init(self, stream=stream)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.address)


_i8, _i32, _i64, _f32 = torch.int8, torch.int32, torch.int64, torch.float32
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _device() -> int:
    try:
        return _current_device()
    except RuntimeError:        # no GPU: every tensor is refused
        return 0


def _raw_stream(stream, dev: int) -> int:
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _refuse(dev: int, ws, *tensors):
    """Raises for the first tensor (name, tensor, dtype, shape with -1 for any size, "strided"
    where its rows may be) that is not what a call takes, or for a workspace elsewhere.  The
    calls test all of them in one expression first, and come here only to name the one at
    fault: a call's checks are much of what a small call costs on the host."""
    for name, t, dtype, shape, *strided in tensors:
        if t is None:
            continue
        if t.dtype != dtype:
            raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
        if t.dim() != len(shape) or any(w not in (-1, g) for w, g in zip(shape, t.shape)):
            raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name}: liblime takes tensors of the current device")
        if not strided and not t.is_contiguous():
            raise ValueError(f"{name}: liblime takes contiguous tensors")
    if ws is not None and ws.device != dev:
        raise ValueError("workspace: liblime takes tensors of the current device")


def _row_dtype(dims):
    return torch.bfloat16 if dims.dtype == LIME_BF16 else torch.float32


def _pitch(name: str, t: torch.Tensor, heads: int, dh: int) -> int:
    """Elements between the rows of t [n, heads, dh], whose heads have to be contiguous."""
    ld, sh, sd = t.stride()
    if (sd != 1 or (sh != dh and heads > 1)) and t.shape[0] > 0:
        raise ValueError(f"{name}: the heads of a row have to be contiguous")
    return ld if t.shape[0] > 1 else heads * dh     # one row has no pitch


def _check_pool(dims, dev, k_cache, v_cache, scale):
    shape = (dims.n_blocks, dims.Hkv, dims.block, dims.dh)
    if not (k_cache.dtype is _i8 and v_cache.dtype is _i8 and scale.dtype is _f32
            and k_cache.shape == shape and v_cache.shape == shape
            and scale.shape == (shape[0], shape[1], 2) and k_cache.get_device() == dev
            and v_cache.get_device() == dev and scale.get_device() == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous() and scale.is_contiguous()):
        _refuse(dev, None, ("k_cache", k_cache, _i8, shape), ("v_cache", v_cache, _i8, shape),
                ("scale", scale, _f32, (shape[0], shape[1], 2)))


def lime_kv_workspace_init(ws: KvWorkspace, stream=None):
    dev = _device()
    _refuse(dev, ws)            # another device's work is not ordered behind this one's stream
    rc = _lib.lime_kv_workspace_init(ws.address, ws.nbytes, _raw_stream(stream, dev))
    if rc:
        raise LimeError("lime_kv_workspace_init", rc)


def lime_kv_reserve(dims, lens, new_offsets, block_table, free_blocks, n_free, lens_out,
                    n_free_out, slot_map, ws: KvWorkspace, stream=None):
    B, dev = lens.shape[0], _device()
    n, cap = slot_map.shape[0], free_blocks.shape[0]
    if not (lens.dtype is _i32 and new_offsets.dtype is _i64 and block_table.dtype is _i32
            and free_blocks.dtype is _i32 and n_free.dtype is _i32 and lens_out.dtype is _i32
            and n_free_out.dtype is _i32 and slot_map.dtype is _i64 and lens.dim() == 1
            and new_offsets.shape == (B + 1,) and block_table.shape == (B, dims.max_blocks)
            and n_free.shape == (1,) and lens_out.shape == (B,) and n_free_out.shape == (1,)
            and lens.get_device() == dev and new_offsets.get_device() == dev
            and block_table.get_device() == dev and free_blocks.get_device() == dev
            and n_free.get_device() == dev and lens_out.get_device() == dev
            and n_free_out.get_device() == dev and slot_map.get_device() == dev
            and lens.is_contiguous() and new_offsets.is_contiguous()
            and block_table.is_contiguous() and free_blocks.is_contiguous()
            and lens_out.is_contiguous() and slot_map.is_contiguous() and ws.device == dev
            and slot_map.dim() == 1 and free_blocks.dim() == 1):
        _refuse(dev, ws, ("lens", lens, _i32, (B,)), ("new_offsets", new_offsets, _i64, (B + 1,)),
                ("block_table", block_table, _i32, (B, dims.max_blocks)),
                ("free_blocks", free_blocks, _i32, (-1,)), ("n_free", n_free, _i32, (1,)),
                ("lens_out", lens_out, _i32, (B,)), ("n_free_out", n_free_out, _i32, (1,)),
                ("slot_map", slot_map, _i64, (-1,)))
    rc = _lib.lime_kv_reserve(
        dims, B, lens.data_ptr(), new_offsets.data_ptr(), n, block_table.data_ptr(),
        free_blocks.data_ptr(), cap, n_free.data_ptr(), lens_out.data_ptr(),
        n_free_out.data_ptr(), slot_map.data_ptr(), ws.address, ws.nbytes, _raw_stream(stream, dev))
    if rc:
        raise LimeError("lime_kv_reserve", rc)


def lime_kv_release(dims, lens, keep: Optional[torch.Tensor], block_table, free_blocks, n_free,
                    lens_out, n_free_out, ws: KvWorkspace, stream=None):
    B, dev = lens.shape[0], _device()
    _refuse(dev, ws, ("lens", lens, _i32, (B,)), ("keep", keep, _i32, (B,)),
            ("block_table", block_table, _i32, (B, dims.max_blocks)),
            ("free_blocks", free_blocks, _i32, (-1,)), ("n_free", n_free, _i32, (1,)),
            ("lens_out", lens_out, _i32, (B,)), ("n_free_out", n_free_out, _i32, (1,)))
    rc = _lib.lime_kv_release(
        dims, B, lens.data_ptr(), None if keep is None else keep.data_ptr(),
        block_table.data_ptr(), free_blocks.data_ptr(), free_blocks.shape[0], n_free.data_ptr(),
        lens_out.data_ptr(), n_free_out.data_ptr(), ws.address, ws.nbytes,
        _raw_stream(stream, dev))
    if rc:
        raise LimeError("lime_kv_release", rc)


def lime_kv_append(dims, K, V, slot_map, k_cache, v_cache, scale, ws: KvWorkspace, stream=None):
    """K, V [n, Hkv, dh] with any row pitch; slot_map int64 [n]."""
    n, dev, dt = slot_map.shape[0], _device(), _row_dtype(dims)
    shape = (n, dims.Hkv, dims.dh)
    if not (K.dtype is dt and V.dtype is dt and slot_map.dtype is _i64 and K.shape == shape
            and V.shape == shape and slot_map.shape == (n,) and K.get_device() == dev
            and V.get_device() == dev and slot_map.get_device() == dev
            and slot_map.is_contiguous() and ws.device == dev):
        _refuse(dev, ws, ("slot_map", slot_map, _i64, (-1,)), ("K", K, dt, shape, "strided"),
                ("V", V, dt, shape, "strided"))
    ldk, ldv = _pitch("K", K, shape[1], shape[2]), _pitch("V", V, shape[1], shape[2])
    _check_pool(dims, dev, k_cache, v_cache, scale)
    rc = _lib.lime_kv_append(
        dims, K.data_ptr(), ldk, V.data_ptr(), ldv, n, slot_map.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), scale.data_ptr(), ws.address, ws.nbytes,
        _raw_stream(stream, dev))
    if rc:
        raise LimeError("lime_kv_append", rc)


def lime_kv_attention(dims, Q, q_offsets, block_table, lens, k_cache, v_cache, scale, O, lse,
                      ws: KvWorkspace, sm_scale: Optional[float] = None, causal: bool = False,
                      stream=None):
    """Q [n, Hq, dh] with any row pitch; lse fp32 [n, Hq] or None; sm_scale 1/sqrt(dh) if None."""
    B, n, dev, dt = lens.shape[0], Q.shape[0], _device(), _row_dtype(dims)
    shape = (n, dims.Hq, dims.dh)
    if not (Q.dtype is dt and O.dtype is dt and q_offsets.dtype is _i64
            and block_table.dtype is _i32 and lens.dtype is _i32 and Q.shape == shape
            and O.shape == shape and lens.dim() == 1 and q_offsets.shape == (B + 1,)
            and block_table.shape == (B, dims.max_blocks)
            and Q.get_device() == dev and O.get_device() == dev and q_offsets.get_device() == dev
            and block_table.get_device() == dev and lens.get_device() == dev
            and O.is_contiguous() and q_offsets.is_contiguous() and block_table.is_contiguous()
            and lens.is_contiguous() and ws.device == dev
            and (lse is None or (lse.dtype is _f32 and lse.shape == shape[:2]
                                 and lse.get_device() == dev and lse.is_contiguous()))):
        _refuse(dev, ws, ("q_offsets", q_offsets, _i64, (B + 1,)),
                ("block_table", block_table, _i32, (B, dims.max_blocks)),
                ("lens", lens, _i32, (B,)), ("O", O, dt, shape), ("lse", lse, _f32, shape[:2]),
                ("Q", Q, dt, shape, "strided"))
    ldq = _pitch("Q", Q, shape[1], shape[2])
    _check_pool(dims, dev, k_cache, v_cache, scale)
    rc = _lib.lime_kv_attention(
        dims, B, Q.data_ptr(), ldq, q_offsets.data_ptr(), n, block_table.data_ptr(),
        lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), scale.data_ptr(),
        1.0 / math.sqrt(dims.dh) if sm_scale is None else sm_scale, 1 if causal else 0,
        O.data_ptr(), None if lse is None else lse.data_ptr(), ws.address, ws.nbytes,
        _raw_stream(stream, dev))
    if rc:
        raise LimeError("lime_kv_attention", rc)


class HistoryCache:
    """The cache of a serving program with B request rows: pool, block table, free stack.

    ``append`` finds room for new rows and writes them, ``attend`` lets query
    rows attend over everything cached, ``release`` shortens requests.  Calls
    are asynchronous on the current stream and belong on one stream.  The
    library's calls read lengths and stack height from one buffer and write
    another, which is then copied back: ``lens`` and ``n_free`` stay where they
    are, so a captured call works on the cache as it stands at each replay.
    ``max_q`` is the most query rows that a captured ``attend`` may have; an eager
    one with more raises it."""

    def __init__(self, dims: lime_kv_dims, B: int, max_q: int = 0, device="cuda"):
        self.dims, self.B = dims, B
        new = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device=device)
        shape = (dims.n_blocks, dims.Hkv, dims.block, dims.dh)
        self.k, self.v = (torch.empty(shape, dtype=torch.int8, device=device) for _ in range(2))
        self.scale = torch.empty(dims.n_blocks, dims.Hkv, 2, device=device)
        self.table = new(B, dims.max_blocks) - 1
        self.free = torch.arange(dims.n_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        self._state, self._next = new(B + 1), new(B + 1)    # lengths, then the stack's height
        self._state[B] = dims.n_blocks
        self.lens, self.n_free = self._state[:B], self._state[B:]
        self._lens, self._n_free = self._next[:B], self._next[B:]
        # one workspace for the cache's life: a captured call keeps writing into it
        self.ws = KvWorkspace(dims, B, max(1, max_q), device=device)
        self.max_q = max_q

    def _advance(self):
        self._state.copy_(self._next)

    def append(self, K: torch.Tensor, V: torch.Tensor, new_offsets: torch.Tensor) -> torch.Tensor:
        """Caches K, V [n, Hkv, dh], request u's rows at [new_offsets[u], new_offsets[u+1]);
        returns the slots (-1: no room)."""
        slots = torch.empty(K.shape[0], dtype=torch.int64, device=K.device)
        lime_kv_reserve(self.dims, self.lens, new_offsets, self.table, self.free, self.n_free,
                        self._lens, self._n_free, slots, self.ws)
        lime_kv_append(self.dims, K, V, slots, self.k, self.v, self.scale, self.ws)
        self._advance()             # a refused call leaves the lengths and the stack as they were
        return slots

    def attend(self, Q: torch.Tensor, q_offsets: torch.Tensor, causal: bool = False,
               sm_scale: Optional[float] = None, lse: Optional[torch.Tensor] = None):
        """Attention of Q [n, Hq, dh] over the cached rows; returns O [n, Hq, dh]."""
        if Q.shape[0] > self.max_q:
            if torch.cuda.is_current_stream_capturing():
                raise ValueError("Q: more rows than max_q, the most that a captured call may have")
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
        _refuse(_device(), self.ws)
        return lime_get_status(self.ws, stream)
