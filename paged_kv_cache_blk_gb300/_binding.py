"""ctypes binding of libpkv: argument marshalling only.

Each function has the name of the C call without the ``pkv_`` prefix, takes
torch tensors, passes their device pointers and the current torch stream to
the library, and raises :class:`PkvError` on any status other than
``PKV_OK``.  Every step of the path runs in the library's CUDA kernels; there
is no Python or CPU fallback, and a missing library is an error.
"""

from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence, Tuple

import numpy as np
import torch

from . import build as _build

_STATUS = {
    0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_CAPACITY", 3: "PKV_ERR_UNSUPPORTED",
    4: "PKV_ERR_WORKSPACE", 5: "PKV_ERR_INDEX", 6: "PKV_ERR_CUDA", 7: "PKV_ERR_TIMEOUT",
    8: "PKV_ERR_NO_BLOCKS",
}
STATUS_CODES = {v: k for k, v in _STATUS.items()}
_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.uint8: 2}


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        self.name = _STATUS.get(status, str(status))
        super().__init__(f"{where}: {self.name} ({message})")


class _PoolStruct(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("num_blocks", ctypes.c_int64),
        ("num_layers", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class _RopeStruct(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("attn_scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("step", ctypes.c_uint64 * 128),
    ]


_lib = None
_P, _I32, _I64, _F32, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
_F64 = ctypes.c_double
_SIGS = {
    "pkv_build_slot_mapping": (_I32, [_P, _P, _I32, _P, _I32, _P, _P, _I64, _P, _P]),
    "pkv_write_slots": (_I32, [_P, _I32, _P, _P, _P, _I64, _P]),
    "pkv_append_tokens": (_I32, [_P, _I32, _P, _I32, _P, _I32, _P, _P, _I64, _P, _P, _P, _P]),
    "pkv_rope_init": (_I32, [_P, _I32, _I32, _F64, _I32, _F64, _F64, _F64, _F64]),
    "pkv_rope_init_freqs": (_I32, [_P, _I32, _I32, _P, _F64]),
    "pkv_rope_append": (_I32, [_P, _I32, _P, _P, _I32, _P, _I32, _P, _P, _P, _I64, _P, _I64, _I32,
                               _P, _I64, _P, _I64, _P, _I64, _P, _P]),
    "pkv_update_block_bounds": (_I32, [_P, _I32, _P, _I32, _P, _P, _P, _I32, _P, _P, _P]),
    "pkv_select_blocks": (_I32, [_P, _I32, _P, _P, _P, _I32, _P, _I32, _P, _I32, _P, _P, _I32,
                                 _I32, _I32, _I32, _P, _P, _P]),
    "pkv_decode_attention_sparse": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _I32, _P, _P,
                                           _I32, _P, _I32, _P, _P]),
    "pkv_decode_attention_window": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _I32, _I32,
                                           _I32, _P, _P]),
    "pkv_prefill_attention_window": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _P, _I32,
                                            _I64, _I32, _I32, _I32, _P, _P]),
    "pkv_decode_tree_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "pkv_decode_attention_tree": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _P, _I32,
                                         _I64, _I32, _P, _I32, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "pkv_accept_tokens": (_I32, [_P, _I32, _P, _I32, _P, _P, _P, _I32, _P, _I32, _P, _P]),
    "pkv_gather": (_I32, [_P, _I32, _P, _I32, _P, _P, _I32, _P, _I64, _P, _P, _P]),
    "pkv_decode_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "pkv_decode_attention": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _I32, _P, _P,
                                    _SZ, _P]),
    "pkv_decode_attention_static": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _I32,
                                           _P, _P]),
    "pkv_decode_shared_prefix_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "pkv_decode_attention_shared_prefix": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P,
                                                  _I32, _I32, _P, _P, _SZ, _P]),
    "pkv_decode_step": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _I32, _P, _P, _P, _P,
                               _SZ, _P]),
    "pkv_copy_blocks": (_I32, [_P, _I32, _P, _P, _I32, _P]),
    "pkv_swap_out": (_I32, [_P, _I32, _P, _I32, _P, _P, _SZ, _P]),
    "pkv_swap_in": (_I32, [_P, _I32, _P, _I32, _P, _P, _SZ, _P]),
    "pkv_prefill_attention": (_I32, [_P, _I32, _P, _I32, _F32, _P, _I32, _P, _P, _P, _I32, _I64,
                                      _I32, _P, _P]),
    "pkv_set_decode_ctas": (_I32, [_I32]),
    "pkv_set_decode_events": (_I32, [_P, _P]),
    "pkv_set_validate": (_I32, [_I32]),
    "pkv_set_wait_limit_ns": (_I32, [ctypes.c_uint64]),
    "pkv_get_wait_limit_ns": (ctypes.c_uint64, []),
    "pkv_set_debug_skip_fill": (_I32, [_I32]),
    "pkv_set_debug_window_path": (_I32, [_I32]),
    "pkv_get_validate": (_I32, []),
    "pkv_device_error": (_I32, [ctypes.POINTER(ctypes.c_int32), _I32]),
    "pkv_alloc_create": (_I32, [_I64, _I32, _P, ctypes.POINTER(ctypes.c_void_p)]),
    "pkv_alloc_destroy": (_I32, [_P]),
    "pkv_alloc_num_free": (_I64, [_P]),
    "pkv_alloc_ref_count": (_I32, [_P, _I64]),
    "pkv_alloc_blocks": (_I32, [_P, _I64, _P]),
    "pkv_alloc_inc_ref": (_I32, [_P, _I32]),
    "pkv_alloc_dec_ref": (_I32, [_P, _I32]),
    "pkv_seq_new": (_I32, [_P, _I64, _I32]),
    "pkv_seq_share": (_I32, [_P, _I64, _P, _I32, _I64]),
    "pkv_seq_append": (_I32, [_P, _I64, _I64, _P, _P, _P, _P]),
    "pkv_seq_append_batch": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P]),
    "pkv_seq_fork": (_I32, [_P, _I64, _I64]),
    "pkv_seq_free": (_I32, [_P, _I64]),
    "pkv_seq_info": (_I32, [_P, _I64, _P, _P, _P]),
    "pkv_seq_tables": (_I32, [_P, _P, _I32, _I32, _P, _P, _P]),
    "pkv_alloc_stats": (_I32, [_P, _P, _P, _P]),
    "pkv_status_string": (ctypes.c_char_p, [_I32]),
    "pkv_version": (_I32, []),
}


def library_path() -> str:
    return _build.LIB


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpkv.so (built by ``build()``); raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"libpkv is not built ({p} missing): run __graft_entry__.build() "
                           "or python -m paged_kv_cache_blk_gb300.build")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != 0:
        msg = load().pkv_status_string(status).decode()
        raise PkvError(status, where, msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The handle alone, where torch offers it (1.8 us less a call): torch.cuda.current_stream
# builds a Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# (a pool lies on the device: torch is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(dev: torch.device) -> int:
    if dev.index is None:
        raise ValueError(f"the pool is on {dev}, not on a CUDA device")
    if _raw_stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev.index)


def int8_row_bytes(num_kv_heads: int, head_dim: int) -> int:
    """Bytes of one token row of an int8 pool (PKV_I8 in include/pkv.h)."""
    return num_kv_heads * head_dim + (4 * num_kv_heads + 15) // 16 * 16


class Pool:
    """K and V block pools ``[num_blocks, num_layers, block_size, num_kv_heads,
    head_dim]`` on one CUDA device, as the library's pool descriptor.  An int8
    pool is a pair of uint8 tensors ``[num_blocks, num_layers, block_size, R]``
    (R = :func:`int8_row_bytes`) with ``num_kv_heads`` and ``head_dim`` given."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 num_kv_heads: Optional[int] = None, head_dim: Optional[int] = None):
        if k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
            raise ValueError("k_cache and v_cache must have the same shape and dtype")
        if not k_cache.is_contiguous() or not v_cache.is_contiguous():
            raise ValueError("pools must be contiguous tensors")
        if k_cache.dtype not in _DTYPE:
            raise ValueError(f"unsupported pool dtype {k_cache.dtype}")
        if k_cache.dtype == torch.uint8:
            if k_cache.dim() != 4 or num_kv_heads is None or head_dim is None:
                raise ValueError("int8 pools are [N, L, bs, R] uint8 tensors with "
                                 "num_kv_heads and head_dim given")
            if k_cache.shape[3] != int8_row_bytes(num_kv_heads, head_dim):
                raise ValueError("int8 pool rows do not match num_kv_heads and head_dim")
            N, L, bs = k_cache.shape[:3]
            H, D = num_kv_heads, head_dim
        else:
            if k_cache.dim() != 5:
                raise ValueError("pools must be contiguous [N, L, bs, Hkv, D] tensors")
            N, L, bs, H, D = k_cache.shape
        self.k_cache, self.v_cache = k_cache, v_cache
        self.struct = _PoolStruct(k_cache.data_ptr(), v_cache.data_ptr(), N, L, bs, H, D,
                                  _DTYPE[k_cache.dtype])
        self.device = k_cache.device
        self.num_blocks, self.num_layers, self.block_size = N, L, bs
        self.num_kv_heads, self.head_dim = H, D
        self.dtype = k_cache.dtype
        # type of q, out and new rows
        self.row_dtype = torch.bfloat16 if k_cache.dtype == torch.uint8 else k_cache.dtype
        self.ref = ctypes.byref(self.struct)
        self.index = k_cache.get_device()


class _NoSwitch:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NO_SWITCH = _NoSwitch()


def _dev(pool: Pool):
    """Make the pool's device current for the call (no-op when it already is)."""
    idx = pool.device.index
    if idx is None or idx == _current_device():
        return _NO_SWITCH
    return torch.cuda.device(pool.device)


def build_slot_mapping(pool: Pool, block_tables: torch.Tensor, offsets: Optional[torch.Tensor],
                       token_seq: torch.Tensor, token_pos: torch.Tensor,
                       slot_mapping: torch.Tensor) -> torch.Tensor:
    """Fill ``slot_mapping`` (int64 [T]) from (sequence, position) pairs."""
    lib = load()
    B = block_tables.shape[0]
    with _dev(pool):
        st = lib.pkv_build_slot_mapping(pool.ref, _ptr(block_tables), block_tables.shape[1],
                                        _ptr(offsets), B, _ptr(token_seq), _ptr(token_pos),
                                        token_seq.numel(), _ptr(slot_mapping),
                                        _stream(pool.device))
    _check(st, "pkv_build_slot_mapping")
    return slot_mapping


def write_slots(pool: Pool, layer: int, k_new: torch.Tensor, v_new: torch.Tensor,
                slot_mapping: torch.Tensor) -> None:
    """Scatter ``k_new``/``v_new`` ([T, Hkv, D]) into the pools at the slots."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_write_slots(pool.ref, layer, _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                 slot_mapping.numel(), _stream(pool.device))
    _check(st, "pkv_write_slots")


def append_tokens(pool: Pool, layer: int, block_tables: torch.Tensor,
                  offsets: Optional[torch.Tensor], token_seq: torch.Tensor,
                  token_pos: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  slot_mapping: Optional[torch.Tensor] = None) -> None:
    """Slot mapping and scatter in one call: rows of ``k_new``/``v_new``
    ([T, Hkv, D]) go to the slots of (token_seq, token_pos); the slots are
    also written to ``slot_mapping`` (int64 [T]) when given."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_append_tokens(pool.ref, layer, _ptr(block_tables), block_tables.shape[1],
                                   _ptr(offsets), block_tables.shape[0], _ptr(token_seq),
                                   _ptr(token_pos), token_seq.numel(), _ptr(k_new), _ptr(v_new),
                                   _ptr(slot_mapping), _stream(pool.device))
    _check(st, "pkv_append_tokens")


class Rope:
    """Rotary schedule of a model (``pkv_rope`` in include/pkv.h): the first
    ``rotary_dim`` dims of a head turn, in pairs (i, i + rotary_dim / 2) or,
    ``interleaved``, (2 i, 2 i + 1).  ``scaling`` for long contexts is None,
    ``"linear"``, ``"base"`` or ``"by_parts"`` (with ``factor``, and for the
    last ``original_len``, ``turns_fast``, ``turns_slow``).  Any other
    schedule, such as the ramp of ``by_parts`` with another factor on cos and
    sin, is given as ``inv_freq`` (radians per token) and ``attn_scale`` (that
    factor), without ``scaling`` and ``factor``."""

    _SCALING = {None: 0, "linear": 1, "base": 2, "by_parts": 3}

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0, original_len: float = 0.0,
                 turns_fast: float = 32.0, turns_slow: float = 1.0,
                 inv_freq: Optional[Sequence[float]] = None, attn_scale: float = 1.0):
        lib = load()
        self.struct = _RopeStruct()
        self.ref = ctypes.byref(self.struct)
        if inv_freq is not None:
            if scaling is not None or factor != 1.0:
                raise ValueError("inv_freq takes the place of a schedule: scaling and factor do "
                                 "not go with it")
            f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
            if f.shape != (rotary_dim // 2,):
                raise ValueError("inv_freq must have rotary_dim / 2 entries")
            _check(lib.pkv_rope_init_freqs(self.ref, rotary_dim, int(bool(interleaved)),
                                           f.ctypes.data, float(attn_scale)),
                   "pkv_rope_init_freqs")
        else:
            if scaling not in self._SCALING:
                raise ValueError(f"unknown rotary scaling {scaling!r}")
            if attn_scale != 1.0:
                raise ValueError("attn_scale goes with inv_freq")
            _check(lib.pkv_rope_init(self.ref, rotary_dim, int(bool(interleaved)), float(base),
                                     self._SCALING[scaling], float(factor), float(original_len),
                                     float(turns_fast), float(turns_slow)), "pkv_rope_init")
        self.rotary_dim, self.interleaved = rotary_dim, bool(interleaved)
        self.attn_scale = float(self.struct.attn_scale)


_INT32, _BF16, _U8 = torch.int32, torch.bfloat16, torch.uint8


# The checks below run on every call and a call's kernels may take a few
# microseconds, so each reads a tensor's properties once and compares whole
# tuples.
def _index(t: Optional[torch.Tensor], pool: Pool, name: str, ndim: int) -> Optional[int]:
    """Pointer of a contiguous int32 index tensor on the pool's device."""
    if t is None:
        return None
    if t.dtype is not _INT32 or t.get_device() != pool.index or t.dim() != ndim \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {ndim} dimension(s) on "
                         f"{pool.device}")
    return t.data_ptr()


def _heads_of(q: torch.Tensor) -> int:
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], not {list(q.shape)}")
    return q.shape[1]


def _rows_of(t: torch.Tensor, pool: Pool, name: str, shape: Tuple[int, int, int]) -> int:
    """Elements between tokens of a [tokens, heads, head_dim] tensor in the
    pool's row type, the heads of a token consecutive."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype is not pool.row_dtype or t.get_device() != pool.index:
        raise ValueError(f"{name} must be {pool.row_dtype} on {pool.device}")
    tokens, heads, d = shape
    st, sh, sd = t.stride()
    if sd != 1 or (sh != d and heads > 1):
        raise ValueError(f"the heads of a token of {name} must be consecutive")
    return st if tokens > 1 else heads * d


def rope_append(pool: Pool, layer: int, rope: Rope, block_tables: torch.Tensor,
                offsets: Optional[torch.Tensor], token_seq: torch.Tensor, token_pos: torch.Tensor,
                q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                q_out: Optional[torch.Tensor], rope_pos: Optional[torch.Tensor] = None,
                slot_mapping: Optional[torch.Tensor] = None) -> None:
    """Rotary positions and append in one pass: ``q`` ([T, Hq, D]) turned into
    ``q_out`` (which may be ``q``), ``k_new`` ([T, Hkv, D]) turned and stored
    with ``v_new`` at the slots of (token_seq, token_pos).  The angle's
    position is ``rope_pos`` where given, else ``token_pos``.  Tokens of q,
    k_new, v_new and q_out may lie apart (slices of one projection)."""
    lib = load()
    T, = token_seq.shape
    B, mb = block_tables.shape
    bt, offs = _index(block_tables, pool, "block_tables", 2), _index(offsets, pool, "offsets", 1)
    seq, pos = _index(token_seq, pool, "token_seq", 1), _index(token_pos, pool, "token_pos", 1)
    rpos = _index(rope_pos, pool, "rope_pos", 1)
    if token_pos.shape[0] != T or (rope_pos is not None and rope_pos.shape[0] != T):
        raise ValueError("token_seq, token_pos and rope_pos must have the same length")
    if offsets is not None and offsets.shape[0] != B:
        raise ValueError("offsets must have one entry per row of block_tables")
    if slot_mapping is not None and (slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T
                                     or slot_mapping.device != pool.device
                                     or not slot_mapping.is_contiguous()):
        raise ValueError("slot_mapping must be a contiguous int64 tensor with an entry per token")
    H, D = pool.num_kv_heads, pool.head_dim
    hq = qs = qos = 0
    qp = qop = None
    if q is not None and q_out is not None:
        hq = _heads_of(q)
        qs, qos = _rows_of(q, pool, "q", (T, hq, D)), _rows_of(q_out, pool, "q_out", (T, hq, D))
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out go together")
    ks, vs = _rows_of(k_new, pool, "k_new", (T, H, D)), _rows_of(v_new, pool, "v_new", (T, H, D))
    with _dev(pool):
        st = lib.pkv_rope_append(pool.ref, layer, rope.ref, bt, mb, offs, B, seq, pos, rpos, T, qp,
                                 qs, hq, k_new.data_ptr(), ks, v_new.data_ptr(), vs, qop, qos,
                                 _ptr(slot_mapping), _stream(pool.device))
    _check(st, "pkv_rope_append")


def gather(pool: Pool, layer: int, block_tables: torch.Tensor, seq_lens: torch.Tensor,
           offsets: Optional[torch.Tensor], cu_seqlens: torch.Tensor, k_out: torch.Tensor,
           v_out: torch.Tensor) -> None:
    """Gather every sequence to packed contiguous ``k_out``/``v_out``."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_gather(pool.ref, layer, _ptr(block_tables), block_tables.shape[1],
                            _ptr(seq_lens), _ptr(offsets), seq_lens.numel(), _ptr(cu_seqlens),
                            k_out.shape[0], _ptr(k_out), _ptr(v_out), _stream(pool.device))
    _check(st, "pkv_gather")


def decode_workspace_size(batch: int, num_q_heads: int, head_dim: int,
                          device: Optional[torch.device] = None) -> int:
    lib = load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = lib.pkv_decode_workspace_size(batch, num_q_heads, head_dim)
    if n == 0:
        raise PkvError(1, "pkv_decode_workspace_size", "bad shape or no CUDA device")
    return n


def decode_attention(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     offsets: Optional[torch.Tensor], out: torch.Tensor,
                     workspace: torch.Tensor) -> None:
    """Paged decode attention of ``q`` [B, Hq, D] into ``out`` [B, Hq, D]."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_decode_attention(pool.ref, layer, _ptr(q), q.shape[1], float(scale),
                                      _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
                                      _ptr(offsets), seq_lens.numel(), _ptr(out),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(pool.device))
    _check(st, "pkv_decode_attention")


def decode_shared_prefix_workspace_size(pool: Pool, batch: int, num_q_heads: int,
                                        num_prefix_blocks: int) -> int:
    with _dev(pool):
        return int(load().pkv_decode_shared_prefix_workspace_size(pool.ref, batch, num_q_heads,
                                                                  num_prefix_blocks))


def decode_attention_shared_prefix(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                                   block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                   offsets: Optional[torch.Tensor], num_prefix_blocks: int,
                                   out: torch.Tensor, workspace: torch.Tensor) -> None:
    """Paged decode attention of ``q`` [B, Hq, D] whose sequences share their
    first ``num_prefix_blocks`` table entries: the prefix is read once."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_decode_attention_shared_prefix(
            pool.ref, layer, _ptr(q), q.shape[1], float(scale), _ptr(block_tables),
            block_tables.shape[1], _ptr(seq_lens), _ptr(offsets), seq_lens.numel(),
            int(num_prefix_blocks), _ptr(out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(pool.device))
    _check(st, "pkv_decode_attention_shared_prefix")


def decode_step(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                block_tables: torch.Tensor, seq_lens: torch.Tensor,
                offsets: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                out: torch.Tensor, workspace: torch.Tensor) -> None:
    """One decode step: store each sequence's new K/V row (``k_new``,
    ``v_new`` [B, Hkv, D]) at its last position, then paged decode attention
    of ``q`` [B, Hq, D] into ``out``, in one pass over the pool."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_decode_step(pool.ref, layer, _ptr(q), q.shape[1], float(scale),
                                 _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
                                 _ptr(offsets), seq_lens.numel(), _ptr(k_new), _ptr(v_new),
                                 _ptr(out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(),
                                 _stream(pool.device))
    _check(st, "pkv_decode_step")


def decode_attention_static(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor,
                            offsets: Optional[torch.Tensor], out: torch.Tensor) -> None:
    """Paged decode attention without a workspace argument: the library keeps
    the scratch in its own fixed device array (for callers that cannot
    allocate device memory where they run; shapes beyond the array's size
    raise PKV_ERR_WORKSPACE, and calls that overlap on the GPU race)."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_decode_attention_static(pool.ref, layer, _ptr(q), q.shape[1], float(scale),
                                             _ptr(block_tables), block_tables.shape[1],
                                             _ptr(seq_lens), _ptr(offsets), seq_lens.numel(),
                                             _ptr(out), _stream(pool.device))
    _check(st, "pkv_decode_attention_static")


class BlockBounds:
    """Key bounds of a pool's blocks (include/pkv.h, "Key bounds"): ``codes``
    uint8 [num_blocks, num_layers, Hkv, 2, head_dim] and ``scales`` fp32
    [num_blocks, num_layers, Hkv] on the pool's device."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != torch.uint8 or codes.dim() != 5 or codes.shape[3] != 2:
            raise ValueError("codes must be a uint8 tensor [N, L, Hkv, 2, D]")
        if scales.dtype != torch.float32 or scales.shape != codes.shape[:3]:
            raise ValueError("scales must be a float32 tensor [N, L, Hkv]")
        if codes.device != scales.device or not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous tensors on one device")
        self.codes, self.scales = codes, scales
        # [N, L, Hkv, D] and the device, compared with a pool's by every call
        self.key = (codes.shape[0], codes.shape[1], codes.shape[2], codes.shape[4], codes.device)

    @classmethod
    def for_pool(cls, pool: Pool) -> "BlockBounds":
        """Bounds for every block of ``pool``, not yet filled."""
        shape = (pool.num_blocks, pool.num_layers, pool.num_kv_heads)
        return cls(torch.empty(shape + (2, pool.head_dim), dtype=torch.uint8, device=pool.device),
                   torch.empty(shape, dtype=torch.float32, device=pool.device))


def _bounds_of(bounds: BlockBounds, pool: Pool) -> None:
    if bounds.key != (pool.num_blocks, pool.num_layers, pool.num_kv_heads, pool.head_dim,
                      pool.device):
        raise ValueError("the bounds do not belong to a pool of this shape")


def update_block_bounds(pool: Pool, layer: int, bounds: BlockBounds, block_tables: torch.Tensor,
                        seq_lens: torch.Tensor, offsets: Optional[torch.Tensor],
                        first_pos: Optional[torch.Tensor] = None) -> None:
    """Recompute the key bounds of the blocks that hold positions
    ``first_pos`` (None: 0) .. ``seq_lens`` - 1 of each sequence."""
    lib = load()
    bt, lens = _index(block_tables, pool, "block_tables", 2), _index(seq_lens, pool, "seq_lens", 1)
    offs, first = _index(offsets, pool, "offsets", 1), _index(first_pos, pool, "first_pos", 1)
    B, mb = block_tables.shape
    for t in (seq_lens, offsets, first_pos):
        if t is not None and t.shape[0] != B:
            raise ValueError("seq_lens, offsets and first_pos must have one entry per row of "
                             "block_tables")
    _bounds_of(bounds, pool)
    with _dev(pool):
        st = lib.pkv_update_block_bounds(pool.ref, layer, bt, mb, lens, offs, first, B, bounds.codes.data_ptr(),
                                         bounds.scales.data_ptr(), _stream(pool.device))
    _check(st, "pkv_update_block_bounds")


def _queries(pool: Pool, q: torch.Tensor, block_tables: torch.Tensor,
             offsets: Optional[torch.Tensor], token_seq: torch.Tensor, token_pos: torch.Tensor,
             selected: torch.Tensor):
    """Checks shared by select_blocks and decode_attention_sparse, and their
    arguments from the tables to the query list."""
    T, = token_seq.shape
    B, mb = block_tables.shape
    bt, offs = _index(block_tables, pool, "block_tables", 2), _index(offsets, pool, "offsets", 1)
    seq, pos = _index(token_seq, pool, "token_seq", 1), _index(token_pos, pool, "token_pos", 1)
    sel = _index(selected, pool, "selected", 3)
    if token_pos.shape[0] != T:
        raise ValueError("token_seq and token_pos must have the same length")
    if offsets is not None and offsets.shape[0] != B:
        raise ValueError("offsets must have one entry per row of block_tables")
    t, h, k = selected.shape
    if t != T or h != pool.num_kv_heads:
        raise ValueError(f"selected must be [{T}, {pool.num_kv_heads}, blocks]")
    hq = _heads_of(q)
    if _rows_of(q, pool, "q", (T, hq, pool.head_dim)) != hq * pool.head_dim:
        raise ValueError("q must be contiguous")
    return (bt, mb, offs, B, seq, pos, T), hq, sel, k


def select_blocks(pool: Pool, layer: int, bounds: BlockBounds, q: torch.Tensor,
                  block_tables: torch.Tensor, offsets: Optional[torch.Tensor],
                  token_seq: torch.Tensor, token_pos: torch.Tensor, selected: torch.Tensor,
                  count: torch.Tensor, sink: int = 0, recent: int = 1) -> None:
    """Score the blocks of each query's sequence from ``bounds`` and select
    ``selected.shape[2]`` of them per kv head: table entries into ``selected``
    (int32 [T, Hkv, K], ascending, -1 behind), their number into ``count``
    (int32 [T, Hkv]).  The first ``sink`` and last ``recent`` are always in."""
    lib = load()
    tokens, hq, sel, k = _queries(pool, q, block_tables, offsets, token_seq, token_pos, selected)
    cnt = _index(count, pool, "count", 2)
    if count.shape != (tokens[-1], pool.num_kv_heads):
        raise ValueError("count must be [T, Hkv]")
    _bounds_of(bounds, pool)
    with _dev(pool):
        st = lib.pkv_select_blocks(pool.ref, layer, bounds.codes.data_ptr(),
                                   bounds.scales.data_ptr(), q.data_ptr(), hq, *tokens, k, sink,
                                   recent, sel, cnt, _stream(pool.device))
    _check(st, "pkv_select_blocks")


def decode_attention_sparse(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                            block_tables: torch.Tensor, offsets: Optional[torch.Tensor],
                            token_seq: torch.Tensor, token_pos: torch.Tensor,
                            selected: torch.Tensor, out: torch.Tensor) -> None:
    """Attention of ``q`` ([T, Hq, D]) over the table entries ``selected``
    (int32 [T, Hkv, K], negative ones skipped) of each query's sequence, at
    positions up to ``token_pos``, into ``out``."""
    lib = load()
    tokens, hq, sel, k = _queries(pool, q, block_tables, offsets, token_seq, token_pos, selected)
    if _rows_of(out, pool, "out", (tokens[-1], hq, pool.head_dim)) != hq * pool.head_dim:
        raise ValueError("out must be contiguous")
    with _dev(pool):
        st = lib.pkv_decode_attention_sparse(pool.ref, layer, q.data_ptr(), hq, float(scale),
                                             *tokens, sel, k, out.data_ptr(),
                                             _stream(pool.device))
    _check(st, "pkv_decode_attention_sparse")


def _refuse_none(**tensors: Optional[torch.Tensor]) -> None:
    missing = [name for name, t in tensors.items() if t is None]
    raise ValueError(f"{', '.join(missing)} must be given")


def _sequences(pool: Pool, block_tables: torch.Tensor, seq_lens: torch.Tensor,
               offsets: Optional[torch.Tensor]):
    """Checks of the tables, lengths and offsets of a batch, and their pointers
    and numbers."""
    if block_tables is None or seq_lens is None:
        _refuse_none(block_tables=block_tables, seq_lens=seq_lens)
    bt, lens = _index(block_tables, pool, "block_tables", 2), _index(seq_lens, pool, "seq_lens", 1)
    offs = _index(offsets, pool, "offsets", 1)
    B, mb = block_tables.shape
    if seq_lens.shape[0] != B or (offsets is not None and offsets.shape[0] != B):
        raise ValueError("seq_lens and offsets must have one entry per row of block_tables")
    return bt, mb, lens, offs, B


def _new_tokens(pool: Pool, cu_q: torch.Tensor, batch: int) -> int:
    """Check of where the new tokens of a batch lie, and its pointer."""
    if cu_q is None:
        _refuse_none(cu_q=cu_q)
    if cu_q.dtype is not torch.int64 or cu_q.get_device() != pool.index \
            or cu_q.shape != (batch + 1,) or not cu_q.is_contiguous():
        raise ValueError(f"cu_q must be a contiguous int64 tensor of {batch + 1} entries on "
                         f"{pool.device}")
    return cu_q.data_ptr()


def _attended(pool: Pool, q: torch.Tensor, out: torch.Tensor, rows: Optional[int] = None) -> int:
    """Checks of q and out ([rows, Hq, D], contiguous); the number of heads."""
    if q is None or out is None:
        _refuse_none(q=q, out=out)
    hq = _heads_of(q)
    shape = (q.shape[0] if rows is None else rows, hq, pool.head_dim)
    for t, name in ((q, "q"), (out, "out")):
        if _rows_of(t, pool, name, shape) != hq * pool.head_dim:
            raise ValueError(f"{name} must be contiguous")
    return hq


def decode_attention_window(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor,
                            offsets: Optional[torch.Tensor], window: int, out: torch.Tensor,
                            sink: int = 0) -> None:
    """Decode attention of ``q`` ([B, Hq, D]) into ``out`` over the last
    ``window`` tokens of each sequence and its first ``sink``."""
    lib = load()
    bt, mb, lens, offs, B = _sequences(pool, block_tables, seq_lens, offsets)
    hq = _attended(pool, q, out, B)
    with _dev(pool):
        st = lib.pkv_decode_attention_window(pool.ref, layer, q.data_ptr(), hq, float(scale), bt,
                                             mb, lens, offs, B, window, sink, out.data_ptr(),
                                             _stream(pool.device))
    _check(st, "pkv_decode_attention_window")


def prefill_attention_window(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor,
                             offsets: Optional[torch.Tensor], cu_q: torch.Tensor, max_q_len: int,
                             window: int, out: torch.Tensor, sink: int = 0) -> None:
    """Prefill attention of ``q`` ([T, Hq, D], the last cu_q[b+1]-cu_q[b] tokens
    of each sequence) into ``out``, each token over the last ``window`` tokens
    up to its own and the first ``sink``."""
    lib = load()
    bt, mb, lens, offs, B = _sequences(pool, block_tables, seq_lens, offsets)
    cu = _new_tokens(pool, cu_q, B)
    hq = _attended(pool, q, out)
    with _dev(pool):
        st = lib.pkv_prefill_attention_window(pool.ref, layer, q.data_ptr(), hq, float(scale), bt,
                                              mb, lens, offs, cu, B, q.shape[0],
                                              max_q_len, window, sink, out.data_ptr(),
                                              _stream(pool.device))
    _check(st, "pkv_prefill_attention_window")


def decode_tree_workspace_size(pool: Pool, batch: int, num_q_heads: int, max_q_len: int) -> int:
    with _dev(pool):
        n = int(load().pkv_decode_tree_workspace_size(pool.ref, batch, num_q_heads, max_q_len))
    if n == 0:
        raise PkvError(1, "pkv_decode_tree_workspace_size", "bad shape or no CUDA device")
    return n


def decode_attention_tree(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          offsets: Optional[torch.Tensor], cu_q: torch.Tensor, max_q_len: int,
                          tree_mask: Optional[torch.Tensor], out: torch.Tensor,
                          workspace: torch.Tensor, q_pos: Optional[torch.Tensor] = None,
                          window: int = 0, sink: int = 0) -> None:
    """Attention of the drafted tokens ``q`` ([T, Hq, D], the last
    cu_q[b+1]-cu_q[b] tokens of each sequence, at most ``max_q_len``) into
    ``out``: over their context and, by the bits of ``tree_mask`` (int64 [T,
    words], bit j of a row: sees drafted token j; None: a chain), over one
    another.  ``window`` (0: none) and ``sink`` limit the context around
    ``q_pos`` (int32 [T], positions along the tree)."""
    lib = load()
    bt, mb, lens, offs, B = _sequences(pool, block_tables, seq_lens, offsets)
    cu = _new_tokens(pool, cu_q, B)
    hq = _attended(pool, q, out)
    T, words, mask = q.shape[0], 0, None
    if tree_mask is not None:
        if tree_mask.dtype is not torch.int64 or tree_mask.get_device() != pool.index \
                or tree_mask.dim() != 2 or tree_mask.shape[0] != T \
                or not tree_mask.is_contiguous():
            raise ValueError(f"tree_mask must be a contiguous int64 tensor [{T}, words] on "
                             f"{pool.device}")
        words, mask = tree_mask.shape[1], tree_mask.data_ptr()
        if words == 0:
            raise ValueError("tree_mask must have a word per 64 drafted tokens")
    qp = _index(q_pos, pool, "q_pos", 1)
    if q_pos is not None and (tree_mask is None or q_pos.shape[0] != T):
        raise ValueError("q_pos goes with tree_mask and has one entry per token")
    if T == 0:  # (tensors of no elements have no address)
        words, mask, qp = 0, None, None
    if workspace is None:
        _refuse_none(workspace=workspace)
    if workspace.get_device() != pool.index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {pool.device}")
    with _dev(pool):
        st = lib.pkv_decode_attention_tree(pool.ref, layer, q.data_ptr(), hq, float(scale), bt, mb,
                                           lens, offs, cu, B, T, max_q_len, mask,
                                           words, qp, window, sink, out.data_ptr(),
                                           workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size(),
                                           _stream(pool.device))
    _check(st, "pkv_decode_attention_tree")


def accept_tokens(pool: Pool, layer: int, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                  offsets: Optional[torch.Tensor], cu_q: torch.Tensor, accepted: torch.Tensor,
                  count: torch.Tensor) -> None:
    """Move the K and V rows of the accepted drafted tokens right behind the
    context: ``accepted`` (int32 [B, most]) holds the ``count`` (int32 [B])
    ascending indices of each sequence; one layer or every one (-1)."""
    lib = load()
    if accepted is None or count is None:
        _refuse_none(accepted=accepted, count=count)
    bt, mb, lens, offs, B = _sequences(pool, block_tables, seq_lens, offsets)
    cu = _new_tokens(pool, cu_q, B)
    path, cnt = _index(accepted, pool, "accepted", 2), _index(count, pool, "count", 1)
    if accepted.shape[0] != B or count.shape[0] != B:
        raise ValueError("accepted and count must have one entry per row of block_tables")
    with _dev(pool):
        st = lib.pkv_accept_tokens(pool.ref, layer, bt, mb, lens, offs, cu, B, path,
                                   accepted.shape[1], cnt, _stream(pool.device))
    _check(st, "pkv_accept_tokens")


def copy_blocks(pool: Pool, layer: int, src_blocks: torch.Tensor,
                dst_blocks: torch.Tensor) -> None:
    """Block dst[i] <- block src[i] (K and V), one layer or every layer (-1)."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_copy_blocks(pool.ref, layer, _ptr(src_blocks), _ptr(dst_blocks),
                                 src_blocks.numel(), _stream(pool.device))
    _check(st, "pkv_copy_blocks")


def swap_out(pool: Pool, layer: int, blocks: torch.Tensor, host_k: torch.Tensor,
             host_v: torch.Tensor) -> None:
    """Listed blocks -> page-locked host tensors [n, layers, bs, Hkv, D]."""
    lib = load()
    nbytes = min(host_k.numel(), host_v.numel()) * host_k.element_size()
    with _dev(pool):
        st = lib.pkv_swap_out(pool.ref, layer, _ptr(blocks), blocks.numel(), _ptr(host_k),
                              _ptr(host_v), nbytes, _stream(pool.device))
    _check(st, "pkv_swap_out")


def swap_in(pool: Pool, layer: int, blocks: torch.Tensor, host_k: torch.Tensor,
            host_v: torch.Tensor) -> None:
    """Page-locked host tensors [n, layers, bs, Hkv, D] -> listed blocks."""
    lib = load()
    nbytes = min(host_k.numel(), host_v.numel()) * host_k.element_size()
    with _dev(pool):
        st = lib.pkv_swap_in(pool.ref, layer, _ptr(blocks), blocks.numel(), _ptr(host_k),
                             _ptr(host_v), nbytes, _stream(pool.device))
    _check(st, "pkv_swap_in")


def prefill_attention(pool: Pool, layer: int, q: torch.Tensor, scale: float,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      offsets: Optional[torch.Tensor], cu_q: torch.Tensor, max_q_len: int,
                      out: torch.Tensor) -> None:
    """Causal prefill attention of q [T, Hq, D] (the last cu_q[b+1]-cu_q[b]
    tokens of each sequence) over the paged cache into out [T, Hq, D]."""
    lib = load()
    with _dev(pool):
        st = lib.pkv_prefill_attention(pool.ref, layer, _ptr(q), q.shape[1], float(scale),
                                       _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
                                       _ptr(offsets), _ptr(cu_q), seq_lens.numel(), q.shape[0],
                                       max_q_len, _ptr(out), _stream(pool.device))
    _check(st, "pkv_prefill_attention")


def set_decode_ctas(n: int) -> None:
    _check(load().pkv_set_decode_ctas(n), "pkv_set_decode_ctas")


def set_decode_events(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]) -> None:
    """Have later decode calls record ``start``/``stop`` around the partial
    pass kernel (``None`` stops it).  The events must have been recorded once
    so that torch has created them."""
    a = start.cuda_event if start is not None else None
    b = stop.cuda_event if stop is not None else None
    _check(load().pkv_set_decode_events(a, b), "pkv_set_decode_events")


def set_validate(on: bool) -> None:
    _check(load().pkv_set_validate(1 if on else 0), "pkv_set_validate")


def set_wait_limit_ns(ns: int) -> None:
    """Bound of every device-side wait in nanoseconds (0 = the default)."""
    _check(load().pkv_set_wait_limit_ns(int(ns)), "pkv_set_wait_limit_ns")


def get_wait_limit_ns() -> int:
    return int(load().pkv_get_wait_limit_ns())


def set_debug_skip_fill(mode: int) -> None:
    """Test hook: with 1 the first CTA, with 2 every CTA, of each decode /
    prefill launch leaves its first stage unfilled, so a wait there can only
    give up; 0 turns it off."""
    _check(load().pkv_set_debug_skip_fill(int(mode)), "pkv_set_debug_skip_fill")


def set_debug_window_path(path: int) -> None:
    """Test hook: ``prefill_attention_window`` takes the mma.sync kernel (1) or
    the tcgen05 kernel (2, refused where that cannot) instead of the one that
    its rule chooses (0)."""
    _check(load().pkv_set_debug_window_path(int(path)), "pkv_set_debug_window_path")


def get_validate() -> bool:
    return bool(load().pkv_get_validate())


def device_error(clear: bool = True) -> str:
    """Status name of the sticky device error word (synchronises the device)."""
    s = ctypes.c_int32(0)
    _check(load().pkv_device_error(ctypes.byref(s), 1 if clear else 0), "pkv_device_error")
    return _STATUS[s.value]


def status_string(status: int) -> str:
    return load().pkv_status_string(status).decode()


def version() -> int:
    return load().pkv_version()


class Allocator:
    """Host block allocator of the library (the allocator section of
    include/pkv.h): FIFO free deque, reference counts, per-sequence block
    tables with a first-block offset, copy-on-write on shared blocks."""

    def __init__(self, num_blocks: int, block_size: int,
                 free_order: Optional[Sequence[int]] = None):
        lib = load()
        h = ctypes.c_void_p()
        order = None
        if free_order is not None:
            order = np.ascontiguousarray(np.asarray(free_order, dtype=np.int32))
        _check(lib.pkv_alloc_create(num_blocks, block_size,
                                    None if order is None else order.ctypes.data,
                                    ctypes.byref(h)), "pkv_alloc_create")
        self._h = h
        self._lib = lib
        self.num_blocks, self.block_size = num_blocks, block_size

    def close(self) -> None:
        if self._h:
            self._lib.pkv_alloc_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def num_free(self) -> int:
        return self._lib.pkv_alloc_num_free(self._h)

    def ref_count(self, block: int) -> int:
        return self._lib.pkv_alloc_ref_count(self._h, block)

    def allocate_blocks(self, n: int) -> List[int]:
        out = np.empty(max(n, 1), dtype=np.int32)
        _check(self._lib.pkv_alloc_blocks(self._h, n, out.ctypes.data), "pkv_alloc_blocks")
        return out[:n].tolist()

    def inc_ref(self, block: int) -> None:
        _check(self._lib.pkv_alloc_inc_ref(self._h, block), "pkv_alloc_inc_ref")

    def dec_ref(self, block: int) -> None:
        _check(self._lib.pkv_alloc_dec_ref(self._h, block), "pkv_alloc_dec_ref")

    def seq_new(self, sid: int, offset: int = 0) -> None:
        _check(self._lib.pkv_seq_new(self._h, sid, offset), "pkv_seq_new")

    def seq_share(self, sid: int, blocks: Sequence[int], num_tokens: int) -> None:
        arr = np.ascontiguousarray(np.asarray(blocks, dtype=np.int32))
        _check(self._lib.pkv_seq_share(self._h, sid, arr.ctypes.data if len(arr) else None,
                                       len(arr), num_tokens), "pkv_seq_share")

    def seq_append(self, sid: int, num_tokens: int) -> Tuple[np.ndarray, List[Tuple[int, int]]]:
        slots = np.empty(max(num_tokens, 1), dtype=np.int64)
        src, dst, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.pkv_seq_append(self._h, sid, num_tokens, slots.ctypes.data,
                                        ctypes.byref(src), ctypes.byref(dst), ctypes.byref(n)),
               "pkv_seq_append")
        return slots[:num_tokens], ([(src.value, dst.value)] if n.value else [])

    def seq_append_batch(self, sids: Sequence[int], counts: Optional[Sequence[int]] = None):
        ids = np.ascontiguousarray(np.asarray(sids, dtype=np.int64))
        n = len(ids)
        cnt = None if counts is None else np.ascontiguousarray(np.asarray(counts, dtype=np.int64))
        total = n if cnt is None else int(cnt.sum())
        slots = np.empty(max(total, 1), dtype=np.int64)
        src = np.empty(max(n, 1), dtype=np.int32)
        dst = np.empty(max(n, 1), dtype=np.int32)
        nc = ctypes.c_int32()
        _check(self._lib.pkv_seq_append_batch(self._h, ids.ctypes.data if n else None, n,
                                              None if cnt is None else cnt.ctypes.data,
                                              slots.ctypes.data, src.ctypes.data, dst.ctypes.data,
                                              ctypes.byref(nc)), "pkv_seq_append_batch")
        return slots[:total], list(zip(src[:nc.value].tolist(), dst[:nc.value].tolist()))

    def seq_fork(self, src: int, dst: int) -> None:
        _check(self._lib.pkv_seq_fork(self._h, src, dst), "pkv_seq_fork")

    def seq_free(self, sid: int) -> None:
        _check(self._lib.pkv_seq_free(self._h, sid), "pkv_seq_free")

    def seq_info(self, sid: int) -> Tuple[int, int, int]:
        n, off, nb = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check(self._lib.pkv_seq_info(self._h, sid, ctypes.byref(n), ctypes.byref(off),
                                      ctypes.byref(nb)), "pkv_seq_info")
        return n.value, off.value, nb.value

    def seq_tables(self, sids: Sequence[int], max_blocks: int):
        ids = np.ascontiguousarray(np.asarray(sids, dtype=np.int64))
        B = len(ids)
        tables = np.empty((max(B, 1), max_blocks), dtype=np.int32)
        lens = np.empty(max(B, 1), dtype=np.int32)
        offs = np.empty(max(B, 1), dtype=np.int32)
        _check(self._lib.pkv_seq_tables(self._h, ids.ctypes.data if B else None, B, max_blocks,
                                        tables.ctypes.data, lens.ctypes.data, offs.ctypes.data),
               "pkv_seq_tables")
        return tables[:B], lens[:B], offs[:B]

    def stats(self) -> Tuple[int, int, float]:
        a, u, f = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_double()
        _check(self._lib.pkv_alloc_stats(self._h, ctypes.byref(a), ctypes.byref(u),
                                         ctypes.byref(f)), "pkv_alloc_stats")
        return a.value, u.value, f.value
