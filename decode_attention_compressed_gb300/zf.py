"""Thin Python binding over libzf.so (C ABI in include/zf.h).

Argument marshalling only: torch tensors provide device memory and the current CUDA stream; every
step of encoding, decompression and attention runs in the library's CUDA kernels.  The library is
loaded on first use and a missing library raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libzf.so")

HEAD_DIM = 128
SLOT_BYTES = 784
RAW_BLOCK_BYTES = 1024
DIR_COMPRESSED = -1
DIR_INVALID = -2
ENCODE_FORCE_RAW = 1
DEV_BAD_PAGE_ID, DEV_BAD_RAW_SLOT, DEV_BAD_N_VALID = 0x1, 0x2, 0x4
DEV_BAD_SEQ_LEN, DEV_BAD_DIR, DEV_TIMEOUT, DEV_BAD_SLOT = 0x8, 0x10, 0x20, 0x40
DEV_NOT_FINITE, DEV_CAPACITY, DEV_BAD_DRAFT, DEV_BAD_PROBS = 0x80, 0x100, 0x200, 0x400
DEV_BAD_FORK = 0x800
Q4_RECORD_BYTES = 2304

_c_int32, _c_void_p, _c_size_t, _c_float = ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float


class ZfCacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_pages", _c_int32), ("num_kv_heads", _c_int32), ("head_dim", _c_int32),
        ("page_size", _c_int32), ("num_raw_slots", _c_int32), ("reserved", _c_int32),
        ("k_comp", _c_void_p), ("v_comp", _c_void_p), ("k_raw", _c_void_p), ("v_raw", _c_void_p),
        ("dir", _c_void_p), ("status", _c_void_p),
    ]


class ZfQ4CacheDesc(ctypes.Structure):
    _fields_ = [
        ("num_pages", _c_int32), ("num_kv_heads", _c_int32), ("head_dim", _c_int32), ("page_size", _c_int32),
        ("k_scale", _c_float), ("v_scale", _c_float), ("records", _c_void_p), ("status", _c_void_p),
    ]


class ZfKvStats(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64), ("free_pages", _c_int32), ("free_raw_slots", _c_int32),
        ("active_requests", _c_int32), ("partial_pages", _c_int32), ("pending_pages", _c_int32),
        ("raw_full_pages", _c_int32), ("compressed_pages", _c_int32), ("new_page_capacity", _c_int32),
        ("raw_full_slots", _c_int32),
    ]


_P32 = ctypes.POINTER(_c_int32)

# name -> (restype, argtypes), mirroring include/zf.h
SIGNATURES = {
    "zf_status_string": (ctypes.c_char_p, [_c_int32]),
    "zf_page_head_bytes": (_c_size_t, [_c_int32, _c_int32]),
    "zf_encode_pages": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p, _c_int32, _c_int32, _c_void_p]),
    "zf_append_tokens": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_int32, _c_void_p]),
    "zf_validate_pages": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_void_p, _c_void_p]),
    "zf_slot_is_valid": (_c_int32, [_c_void_p]),
    "zf_decompress": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_void_p, _c_void_p, _c_void_p]),
    "zf_decompress_to_raw": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_void_p, _c_void_p,
                                        _c_void_p]),
    "zf_decode_attn_workspace_size": (_c_size_t, [_c_int32, _c_int32, _c_int32, _c_int32, _c_int32]),
    "zf_decode_attn": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_void_p, _c_int32,
                                  _c_void_p, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "zf_dense_decode_attn": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_void_p,
                                        _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                        _c_void_p]),
    "zf_decode_attn_static": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_void_p,
                                         _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p, _c_void_p]),
    "zf_decode_attn_multi_workspace_size": (_c_size_t, [_c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32]),
    "zf_decode_attn_multi": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                        _c_void_p, _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p, _c_void_p,
                                        _c_size_t, _c_void_p]),
    "zf_decode_attn_multi_kernel": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                               _c_void_p, _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p,
                                               _c_void_p, _c_size_t, _c_int32, _c_void_p]),
    "zf_decode_attn_wait_test": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                            _c_void_p, _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p,
                                            _c_void_p, _c_size_t, _c_int32, ctypes.c_uint64, ctypes.c_uint64,
                                            _c_void_p]),
    "zf_dense_decode_attn_multi": (_c_int32, [ctypes.POINTER(ZfCacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                              _c_void_p, _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p,
                                              _c_void_p, _c_size_t, _c_void_p]),
    "zf_q4_write_tokens": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int32,
                                      _c_void_p]),
    "zf_q4_read_tokens": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_void_p, _c_int32, _c_void_p, _c_void_p,
                                     _c_void_p]),
    "zf_q4_decode_attn_workspace_size": (_c_size_t, [_c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32]),
    "zf_q4_decode_attn": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32, _c_void_p,
                                     _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                     _c_void_p]),
    "zf_q4_decode_attn_wait_test": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                               _c_void_p, _c_int32, _c_void_p, _c_float, _c_void_p, _c_void_p,
                                               _c_void_p, _c_size_t, ctypes.c_uint64, _c_void_p]),
    "zf_q4_chunk_attn_workspace_size": (_c_size_t, [_c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32]),
    "zf_q4_chunk_attn": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32, _c_void_p,
                                    _c_void_p, _c_int32, _c_void_p, _c_float, _c_int32, _c_float, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "zf_q4_chunk_attn_wait_test": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_int32, _c_int32, _c_int32,
                                              _c_void_p, _c_void_p, _c_int32, _c_void_p, _c_float, _c_int32, _c_float,
                                              _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t, ctypes.c_uint64,
                                              _c_void_p]),
    "zf_map_tokens": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_void_p, _c_int32, _c_void_p, _c_void_p]),
    "zf_fork_requests": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int32,
                                    _c_void_p, _c_void_p, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p]),
    "zf_q4_copy_pages": (_c_int32, [ctypes.POINTER(ZfQ4CacheDesc), _c_void_p, _c_void_p, _c_int32, _c_void_p]),
    "zf_release_requests_workspace_size": (_c_size_t, [_c_int32]),
    "zf_release_requests": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                       _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                       _c_void_p]),
    "zf_compact_pages_workspace_size": (_c_size_t, [_c_int32]),
    "zf_compact_pages": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "zf_sample_tokens": (_c_int32, [_c_int32, _c_int32, _c_void_p, _c_int32, ctypes.c_int64, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "zf_verify_drafts": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "zf_verify_mapped_drafts": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                           _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                           _c_void_p]),
    "zf_kv_create": (_c_int32, [_c_int32, _c_int32, _c_int32, _c_int32, _c_int32, _c_int32, ctypes.POINTER(_c_void_p)]),
    "zf_kv_destroy": (None, [_c_void_p]),
    "zf_kv_admit": (_c_int32, [_c_void_p, _c_int32, _c_int32, _P32, _P32, _P32, _P32]),
    "zf_kv_append": (_c_int32, [_c_void_p, _P32, _c_int32, _P32, _P32, _P32]),
    "zf_kv_pending": (_c_int32, [_c_void_p, _P32, _P32, _c_int32, _P32]),
    "zf_kv_reclaim": (_c_int32, [_c_void_p, _P32, _P32, _c_int32]),
    "zf_kv_release": (_c_int32, [_c_void_p, _c_int32]),
    "zf_kv_export": (_c_int32, [_c_void_p, _P32, _P32]),
    "zf_kv_get_stats": (_c_int32, [_c_void_p, ctypes.POINTER(ZfKvStats)]),
    "zf_kv_plan_pages": (_c_int32, [ctypes.c_int64, _c_int32, _c_int32, _c_int32, _P32, _P32]),
}

_LIB = None


class ZfError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """The loaded libzf.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ZfError(f"{LIB_PATH} is missing: build it with `python -m decode_attention_compressed_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _LIB = handle
    return _LIB


def status_string(code: int) -> str:
    return lib().zf_status_string(code).decode()


def _check(name: str, code: int):
    if code != 0:
        raise ZfError(f"{name}: {status_string(code)} ({code})")


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev_i32(x, device):
    return torch.as_tensor(x, dtype=torch.int32, device=device).contiguous()


_BITS16 = (torch.int16, torch.bfloat16)      # BF16 bit patterns, either view


def _count(x) -> int:
    return int(x.numel()) if isinstance(x, torch.Tensor) else len(x)


def _arg(t, name, cache, dtypes, shape=None, min_rows=None):
    """Checks the C ABI cannot make (it sees bare pointers): dtype, device, shape.  `shape` entries
    of None match any size; min_rows bounds the first dimension from below."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    if shape is not None and (t.dim() != len(shape) or
                              any(w is not None and h != w for h, w in zip(t.shape, shape))):
        want = "[" + "][".join("*" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name}: shape {list(t.shape)}, expected {want}")
    if min_rows is not None and (t.dim() < 1 or t.shape[0] < min_rows):
        raise ValueError(f"{name}: {t.shape[0] if t.dim() else 0} rows, at least {min_rows} needed")
    return t.contiguous()


def _result(t, name, cache, shape):
    """An output the kernels write in place: float32, contiguous, exactly `shape`."""
    _arg(t, name, cache, (torch.float32,), shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (it is written in place)")
    return t


def _attn_args(cache, q, page_table, seq_lens, B):
    page_table = _arg(page_table, "page_table", cache, (torch.int32,), (None, None), min_rows=B)
    seq_lens = _arg(seq_lens, "seq_lens", cache, (torch.int32,), (None,), min_rows=B)
    return page_table, seq_lens


class Cache:
    """One layer's paged cache in device memory, laid out as include/zf.h describes.

    k_comp/v_comp: [num_pages][Hkv][P/4 * 784] uint8; k_raw/v_raw: [num_raw][Hkv][P/4 * 512] int16
    (BF16 bits); dir: [num_pages][Hkv] int32; status: one int32 device word.  raw_pool=another
    Cache makes this layer use that cache's raw arrays (one raw pool for all layers, as KvManager
    with num_layers > 1 hands out slots).
    """

    def __init__(self, num_pages, num_kv_heads, page_size, num_raw_slots, device="cuda", compressed=True,
                 raw_pool=None):
        nblk = page_size // 4
        self.num_pages, self.num_kv_heads, self.page_size = num_pages, num_kv_heads, page_size
        self.num_raw_slots = num_raw_slots
        dev = torch.device(device)
        if raw_pool is not None:                   # share another cache's raw arrays (one pool for all layers)
            if (raw_pool.num_kv_heads, raw_pool.page_size, raw_pool.num_raw_slots) != (num_kv_heads, page_size,
                                                                                      num_raw_slots):
                raise ValueError("a shared raw pool must match the kv heads, page size and raw slot count")
        if compressed:
            self.k_comp = torch.empty((num_pages, num_kv_heads, nblk * SLOT_BYTES), dtype=torch.uint8, device=dev)
            self.v_comp = torch.empty_like(self.k_comp)
        else:
            self.k_comp = self.v_comp = None       # dense cache: raw slots only (zf_dense_decode_attn)
        self.dir = torch.full((num_pages, num_kv_heads), DIR_INVALID, dtype=torch.int32, device=dev)
        if raw_pool is not None:
            self.k_raw, self.v_raw = raw_pool.k_raw, raw_pool.v_raw
        else:
            self.k_raw = torch.empty((num_raw_slots, num_kv_heads, nblk * 512), dtype=torch.int16, device=dev)
            self.v_raw = torch.empty_like(self.k_raw)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    @property
    def device(self):
        return self.status.device

    def desc(self) -> ZfCacheDesc:
        return ZfCacheDesc(self.num_pages, self.num_kv_heads, HEAD_DIM, self.page_size, self.num_raw_slots, 0,
                           _ptr(self.k_comp), _ptr(self.v_comp), _ptr(self.k_raw), _ptr(self.v_raw),
                           _ptr(self.dir), _ptr(self.status))

    def status_word(self) -> int:
        return int(self.status.item())

    def stored_bytes(self, num_pages=None) -> int:
        """Bytes the first `num_pages` pages actually occupy (synchronises): every page head costs
        its compressed record or its raw record, plus its directory entry."""
        n = self.num_pages if num_pages is None else num_pages
        nblk = self.page_size // 4
        if self.k_comp is None:
            return n * self.num_kv_heads * 2 * nblk * RAW_BLOCK_BYTES
        d = self.dir[:n].cpu()
        comp = int((d == DIR_COMPRESSED).sum())
        raw = int((d >= 0).sum())
        return 2 * nblk * (comp * SLOT_BYTES + raw * RAW_BLOCK_BYTES) + d.numel() * 4


def encode_pages(cache: Cache, src_k, src_v, page_ids, n_valid, raw_slots=None, force_raw=False, stream=None):
    """Compress (or store raw) pages: src_k/src_v [n][Hkv][P][128] int16 BF16 bits on the device."""
    dev = cache.device
    shape = (None, cache.num_kv_heads, cache.page_size, HEAD_DIM)
    src_k = _arg(src_k, "src_k", cache, _BITS16, shape)
    src_v = _arg(src_v, "src_v", cache, _BITS16, tuple(src_k.shape))
    n = int(src_k.shape[0])
    for name, x in (("page_ids", page_ids), ("n_valid", n_valid), ("raw_slots", raw_slots)):
        if x is not None and _count(x) != n:
            raise ValueError(f"{name}: {_count(x)} entries for {n} pages")
    ids = _dev_i32(page_ids, dev)
    nv = _dev_i32(n_valid, dev)
    rs = _dev_i32(raw_slots, dev) if raw_slots is not None else _dev_i32([-1] * n, dev)
    d = cache.desc()
    code = lib().zf_encode_pages(ctypes.byref(d), _ptr(src_k), _ptr(src_v), _ptr(ids), _ptr(nv), _ptr(rs), n,
                                 ENCODE_FORCE_RAW if force_raw else 0, _stream(stream))
    _check("zf_encode_pages", code)
    return ids, nv, rs          # keep them alive until the stream has consumed them


def append_tokens(cache: Cache, k_tok, v_tok, page_ids, positions, raw_slots, stream=None):
    """zf_append_tokens: k_tok/v_tok [n][Hkv][128] int16 BF16 bits on the device; entry i is token
    positions[i] of page page_ids[i], written into raw slot raw_slots[i] (the page is compressed
    when that token fills it).  Returns the index tensors (keep them alive until the stream has
    consumed them)."""
    dev = cache.device
    k_tok = _arg(k_tok, "k_tok", cache, _BITS16, (None, cache.num_kv_heads, HEAD_DIM))
    v_tok = _arg(v_tok, "v_tok", cache, _BITS16, tuple(k_tok.shape))
    n = int(k_tok.shape[0])
    for name, x in (("page_ids", page_ids), ("positions", positions), ("raw_slots", raw_slots)):
        if _count(x) != n:
            raise ValueError(f"{name}: {_count(x)} entries for {n} tokens")
    ids, pos, rs = _dev_i32(page_ids, dev), _dev_i32(positions, dev), _dev_i32(raw_slots, dev)
    d = cache.desc()
    _check("zf_append_tokens", lib().zf_append_tokens(ctypes.byref(d), _ptr(k_tok), _ptr(v_tok), _ptr(ids), _ptr(pos),
                                                       _ptr(rs), n, _stream(stream)))
    return ids, pos, rs


def validate_pages(cache: Cache, page_ids, stream=None):
    """zf_validate_pages: an int32 device tensor, 1 for each listed page whose stored form has a
    problem (the cache's status word says which kind)."""
    dev = cache.device
    ids = _dev_i32(page_ids, dev)
    bad = torch.zeros(int(ids.numel()), dtype=torch.int32, device=dev)
    d = cache.desc()
    _check("zf_validate_pages", lib().zf_validate_pages(ctypes.byref(d), _ptr(ids), int(ids.numel()), _ptr(bad),
                                                         _stream(stream)))
    return bad


def slot_is_valid(slot) -> bool:
    """zf_slot_is_valid on one 784-byte compressed slot held in host memory (bytes or uint8 array)."""
    buf = (ctypes.c_uint8 * SLOT_BYTES).from_buffer_copy(bytes(slot)[:SLOT_BYTES].ljust(SLOT_BYTES, b"\0"))
    return bool(lib().zf_slot_is_valid(ctypes.addressof(buf)))


def decompress(cache: Cache, page_ids, stream=None):
    dev = cache.device
    ids = _dev_i32(page_ids, dev)
    n = int(ids.numel())
    k = torch.empty((n, cache.num_kv_heads, cache.page_size, HEAD_DIM), dtype=torch.int16, device=dev)
    v = torch.empty_like(k)
    d = cache.desc()
    _check("zf_decompress", lib().zf_decompress(ctypes.byref(d), _ptr(ids), n, _ptr(k), _ptr(v), _stream(stream)))
    return k, v


def decompress_to_raw(cache: Cache, page_ids, dense: Cache, stream=None):
    """zf_decompress_to_raw: page_ids[i] of `cache` into raw slot i of the dense cache `dense`
    (same kv heads and page size, at least len(page_ids) raw slots).  Returns the id tensor (keep it
    alive until the stream has consumed it)."""
    dev = cache.device
    ids = _dev_i32(page_ids, dev)
    n = int(ids.numel())
    if dense.num_kv_heads != cache.num_kv_heads or dense.page_size != cache.page_size or dense.num_raw_slots < n:
        raise ValueError("the dense cache must match the kv heads and page size and hold n raw slots")
    d = cache.desc()
    _check("zf_decompress_to_raw", lib().zf_decompress_to_raw(ctypes.byref(d), _ptr(ids), n, _ptr(dense.k_raw),
                                                               _ptr(dense.v_raw), _stream(stream)))
    return ids


def workspace_size(batch, num_q_heads, num_kv_heads, page_size, max_pages) -> int:
    return int(lib().zf_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, page_size, max_pages))


def new_workspace(nbytes, device="cuda"):
    """A workspace buffer for zf_decode_attn (any contents are fine)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# attention kernels of zf_decode_attn_multi_kernel
KERNELS = {"auto": 0, "warp_mma": 1, "tcgen05": 2}


def _kernel_code(kernel, dense):
    if kernel not in KERNELS:
        raise ValueError(f"kernel must be one of {sorted(KERNELS)}")
    if dense and kernel != "auto":
        raise ValueError("the dense comparator has one kernel (warp MMA)")
    return KERNELS[kernel]


def decode_attn(cache: Cache, q, page_table, seq_lens, scale=None, out=None, lse=None, workspace=None,
                stream=None, dense=False, kernel="auto"):
    """Decode attention over the cache.  q [B][Hq][128] int16 (BF16 bits), page_table [B][max_pages]
    int32, seq_lens [B] int32, all on the device.  Returns (out [B][Hq][128] f32, lse [B][Hq] f32).
    dense=True runs zf_dense_decode_attn on the raw pool (page id = raw slot).  kernel: "auto"
    (zf_decode_attn), or "warp_mma" / "tcgen05" (zf_decode_attn_multi_kernel with one new token)."""
    code = _kernel_code(kernel, dense)
    if code:
        o, l = decode_attn_multi(cache, q[:, None], page_table, seq_lens, scale,
                                 out=None if out is None else out[:, None], lse=None if lse is None else lse[:, None],
                                 workspace=workspace, stream=stream, kernel=kernel)
        return o[:, 0], l[:, 0]
    q = _arg(q, "q", cache, _BITS16, (None, None, HEAD_DIM))
    B, Hq, _ = q.shape
    page_table, seq_lens = _attn_args(cache, q, page_table, seq_lens, B)
    max_pages = int(page_table.shape[1])
    scale = 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale
    dev = cache.device
    out = torch.empty((B, Hq, HEAD_DIM), dtype=torch.float32, device=dev) if out is None else \
        _result(out, "out", cache, (B, Hq, HEAD_DIM))
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else _result(lse, "lse", cache, (B, Hq))
    need = workspace_size(B, Hq, cache.num_kv_heads, cache.page_size, max_pages)
    if workspace is None:
        workspace = new_workspace(need, dev)
    d = cache.desc()
    fn = lib().zf_dense_decode_attn if dense else lib().zf_decode_attn
    code = fn(ctypes.byref(d), _ptr(q), B, Hq, _ptr(page_table), max_pages, _ptr(seq_lens), scale, _ptr(out),
              _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("zf_dense_decode_attn" if dense else "zf_decode_attn", code)
    return out, lse


def dense_decode_attn(cache: Cache, q, page_table, seq_lens, scale=None, **kw):
    return decode_attn(cache, q, page_table, seq_lens, scale, dense=True, **kw)


def workspace_size_multi(batch, tokens, num_q_heads, num_kv_heads, page_size, max_pages) -> int:
    return int(lib().zf_decode_attn_multi_workspace_size(batch, tokens, num_q_heads, num_kv_heads, page_size,
                                                         max_pages))


def decode_attn_multi(cache: Cache, q, page_table, seq_lens, scale=None, out=None, lse=None, workspace=None,
                      stream=None, dense=False, kernel="auto"):
    """zf_decode_attn_multi: T new tokens per request.  q [B][T][Hq][128] int16 (BF16 bits); token t
    of request b attends to positions 0 .. seq_lens[b] - T + t.  Returns (out [B][T][Hq][128] f32,
    lse [B][T][Hq] f32).  dense=True runs zf_dense_decode_attn_multi.  kernel: "auto", "warp_mma" or
    "tcgen05" (zf_decode_attn_multi_kernel)."""
    code = _kernel_code(kernel, dense)
    q = _arg(q, "q", cache, _BITS16, (None, None, None, HEAD_DIM))
    B, T, Hq, _ = q.shape
    page_table, seq_lens = _attn_args(cache, q, page_table, seq_lens, B)
    max_pages = int(page_table.shape[1])
    scale = 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale
    dev = cache.device
    out = torch.empty((B, T, Hq, HEAD_DIM), dtype=torch.float32, device=dev) if out is None else \
        _result(out, "out", cache, (B, T, Hq, HEAD_DIM))
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev) if lse is None else \
        _result(lse, "lse", cache, (B, T, Hq))
    if workspace is None:
        workspace = new_workspace(workspace_size_multi(B, T, Hq, cache.num_kv_heads, cache.page_size, max_pages), dev)
    d = cache.desc()
    args = (ctypes.byref(d), _ptr(q), B, T, Hq, _ptr(page_table), max_pages, _ptr(seq_lens), scale, _ptr(out),
            _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size())
    if code:
        name = "zf_decode_attn_multi_kernel"
        status = lib().zf_decode_attn_multi_kernel(*args, code, _stream(stream))
    else:
        name = "zf_dense_decode_attn_multi" if dense else "zf_decode_attn_multi"
        status = getattr(lib(), name)(*args, _stream(stream))
    _check(name, status)
    return out, lse


def decode_attn_wait_test(cache: Cache, q, page_table, seq_lens, scale=None, kernel="warp_mma", wait_limit_ns=1000000,
                          publish_delay_ns=0, stream=None):
    """zf_decode_attn_wait_test (tests of the failure path): one new token per request, the
    kernel's waits for its metadata warp's items limited to wait_limit_ns and that warp's first
    item published publish_delay_ns late.  Returns (out, lse); with the delay above the limit
    the outputs are not meaningful and the cache's status word gets DEV_TIMEOUT."""
    q = _arg(q, "q", cache, _BITS16, (None, None, HEAD_DIM))
    B, Hq, _ = q.shape
    page_table, seq_lens = _attn_args(cache, q, page_table, seq_lens, B)
    max_pages = int(page_table.shape[1])
    scale = 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale
    dev = cache.device
    out = torch.empty((B, Hq, HEAD_DIM), dtype=torch.float32, device=dev)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    workspace = new_workspace(workspace_size(B, Hq, cache.num_kv_heads, cache.page_size, max_pages), dev)
    d = cache.desc()
    _check("zf_decode_attn_wait_test",
           lib().zf_decode_attn_wait_test(ctypes.byref(d), _ptr(q), B, 1, Hq, _ptr(page_table), max_pages,
                                          _ptr(seq_lens), scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _kernel_code(kernel, False),
                                          int(wait_limit_ns), int(publish_delay_ns), _stream(stream)))
    return out, lse


STATIC_WORKSPACE_BYTES = 32 << 20
ERR_STATIC_WORKSPACE_EXCEEDED = -5
ERR_STATIC_WORKSPACE_UNAVAILABLE = -7


def decode_attn_static(cache: Cache, q, page_table, seq_lens, scale=None, out=None, lse=None, stream=None):
    """zf_decode_attn_static: the same attention without a caller-provided workspace, for callers
    that cannot allocate device memory (the library's 32 MiB static scratch array is used).
    Calls must not overlap on the GPU; the first call on a device must precede any stream capture."""
    q = _arg(q, "q", cache, _BITS16, (None, None, HEAD_DIM))
    B, Hq, _ = q.shape
    page_table, seq_lens = _attn_args(cache, q, page_table, seq_lens, B)
    scale = 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale
    dev = cache.device
    out = torch.empty((B, Hq, HEAD_DIM), dtype=torch.float32, device=dev) if out is None else \
        _result(out, "out", cache, (B, Hq, HEAD_DIM))
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else _result(lse, "lse", cache, (B, Hq))
    d = cache.desc()
    code = lib().zf_decode_attn_static(ctypes.byref(d), _ptr(q), B, Hq, _ptr(page_table), int(page_table.shape[1]),
                                       _ptr(seq_lens), scale, _ptr(out), _ptr(lse), _stream(stream))
    _check("zf_decode_attn_static", code)
    return out, lse


# ------------------------------------------------------------------ the 4-bit cache (zf_q4_*)
def _tensor(t, name, dtypes, device, shape, write=False):
    """`t` checked for dtype, device and exact shape; contiguous (a tensor written in place has to be)."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and t.shape == shape:
        if t.is_contiguous():
            return t
        if not write:
            return t.contiguous()
        raise ValueError(f"{name} must be contiguous (it is written in place)")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name}: shape {list(t.shape)}, expected {list(shape)}")


_I32, _F32 = (torch.int32,), (torch.float32,)


def _on_stream(call):
    """A call given stream= runs with that stream current, so that what it allocates or copies is
    ordered with its kernels."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


def _launch_stream(device) -> int:
    """The current stream; the tensors' device has to be the current one (the kernels take its pointers)."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: a CUDA device is needed")
    current = torch.cuda.current_device()
    if device.index != current:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{current}")
    return torch._C._cuda_getCurrentRawStream(current)


def _tables(page_table, seq_lens, device, B):
    """page_table [>= B][*] and seq_lens [>= B], int32."""
    for t, name, dims in ((page_table, "page_table", 2), (seq_lens, "seq_lens", 1)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.int32:
            raise ValueError(f"{name}: dtype {t.dtype}, expected torch.int32")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the cache on {device}")
        if len(t.shape) != dims:
            raise ValueError(f"{name}: shape {list(t.shape)}, expected {'[*][*]' if dims == 2 else '[*]'}")
        if t.shape[0] < B:
            raise ValueError(f"{name}: {t.shape[0]} rows, at least {B} needed")
    return page_table.contiguous(), seq_lens.contiguous()


# (The calls below also take stream=, a torch.cuda.Stream to run on.)
class Q4Cache:
    """One layer's 4-bit paged cache in device memory (layout and numbers: include/zf.h, zf_q4).

    records: [num_pages][Hkv][P/16][2304] uint8, given or allocated (zeros: every token reads as 0);
    status: one int32 device word.  k_scale / v_scale multiply the stored values (1 suits values up
    to about 2688).  Sizes, scales and tensors are fixed once made.
    """

    def __init__(self, num_pages, num_kv_heads, page_size, device="cuda", k_scale=1.0, v_scale=1.0, records=None):
        shape = (num_pages, num_kv_heads, page_size // 16, Q4_RECORD_BYTES)
        if records is None:
            records = torch.zeros(shape, dtype=torch.uint8, device=torch.device(device))
        else:
            _tensor(records, "records", (torch.uint8,), getattr(records, "device", None), shape, write=True)
        self._sizes = (num_pages, num_kv_heads, page_size, float(k_scale), float(v_scale))
        self._records, self._device = records, records.device
        self._status = torch.zeros(1, dtype=torch.int32, device=records.device)
        self._desc = ZfQ4CacheDesc(num_pages, num_kv_heads, HEAD_DIM, page_size, float(k_scale), float(v_scale),
                                   _ptr(records), _ptr(self._status))
        self._ref = ctypes.byref(self._desc)

    num_pages = property(lambda self: self._sizes[0])
    num_kv_heads = property(lambda self: self._sizes[1])
    page_size = property(lambda self: self._sizes[2])
    k_scale = property(lambda self: self._sizes[3])
    v_scale = property(lambda self: self._sizes[4])
    records = property(lambda self: self._records)
    status = property(lambda self: self._status)
    device = property(lambda self: self._device)

    def desc(self) -> ZfQ4CacheDesc:
        return self._desc

    def status_word(self) -> int:
        return int(self._status.item())

    def stored_bytes(self) -> int:
        return self._records.numel()


def _places(cache, page_ids, positions):
    """Index lists of a call as int32 device tensors of one length."""
    out = []
    for name, x in (("page_ids", page_ids), ("positions", positions)):
        if not (isinstance(x, torch.Tensor) and x.dtype == torch.int32 and x.device == cache._device):
            x = torch.as_tensor(x, dtype=torch.int32, device=cache._device)
        if x.dim() != 1:
            raise ValueError(f"{name}: shape {list(x.shape)}, expected one dimension")
        out.append(x if x.is_contiguous() else x.contiguous())
    if out[0].shape != out[1].shape:
        raise ValueError(f"positions: {out[1].numel()} entries for {out[0].numel()} tokens")
    return out


@_on_stream
def q4_write_tokens(cache: Q4Cache, k_tok, v_tok, page_ids, positions):
    """zf_q4_write_tokens: k_tok/v_tok [n][Hkv][128] int16 BF16 bits (or bfloat16) on the device; entry i
    is token positions[i] of page page_ids[i] (position -1: skipped).  Returns the index tensors (keep
    them alive until the stream has consumed them)."""
    ids, pos = _places(cache, page_ids, positions)
    n = ids.shape[0]
    shape = (n, cache._sizes[1], HEAD_DIM)
    k_tok = _tensor(k_tok, "k_tok", _BITS16, cache._device, shape)
    v_tok = _tensor(v_tok, "v_tok", _BITS16, cache._device, shape)
    s = _launch_stream(cache._device)
    code = lib().zf_q4_write_tokens(cache._ref, k_tok.data_ptr(), v_tok.data_ptr(), ids.data_ptr(), pos.data_ptr(), n, s)
    if code:
        _check("zf_q4_write_tokens", code)
    return ids, pos


@_on_stream
def q4_read_tokens(cache: Q4Cache, page_ids, positions):
    """zf_q4_read_tokens: the values held at the listed places, (k, v) [n][Hkv][128] int16 BF16 bits."""
    ids, pos = _places(cache, page_ids, positions)
    n = ids.shape[0]
    s = _launch_stream(cache._device)
    shape = (n, cache._sizes[1], HEAD_DIM)
    k = torch.empty(shape, dtype=torch.int16, device=cache._device)
    v = torch.empty(shape, dtype=torch.int16, device=cache._device)
    code = lib().zf_q4_read_tokens(cache._ref, ids.data_ptr(), pos.data_ptr(), n, k.data_ptr(), v.data_ptr(), s)
    if code:
        _check("zf_q4_read_tokens", code)
    return k, v


def q4_workspace_size(batch, tokens, num_q_heads, num_kv_heads, page_size, max_pages) -> int:
    return int(lib().zf_q4_decode_attn_workspace_size(batch, tokens, num_q_heads, num_kv_heads, page_size, max_pages))


@_on_stream
def q4_decode_attn(cache: Q4Cache, q, page_table, seq_lens, scale=None, out=None, lse=None, workspace=None):
    """zf_q4_decode_attn: decode attention over the 4-bit cache.  q [B][Hq][128], or [B][T][Hq][128] for T
    new tokens per request (token t attends to positions 0 .. seq_lens[b] - T + t), int16 BF16 bits or
    bfloat16.  Returns (out f32 of q's shape, lse f32 without the last dimension)."""
    dev = cache._device
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    shape = q.shape
    if len(shape) not in (3, 4) or shape[-1] != HEAD_DIM:
        raise ValueError(f"q: shape {list(shape)}, expected [*][*][{HEAD_DIM}] or [*][*][*][{HEAD_DIM}]")
    q = _tensor(q, "q", _BITS16, dev, shape)
    B, T, Hq = (shape[0], 1, shape[1]) if len(shape) == 3 else shape[:3]
    page_table, seq_lens = _tables(page_table, seq_lens, dev, B)
    max_pages = page_table.shape[1]
    out = torch.empty(shape, dtype=torch.float32, device=dev) if out is None else \
        _tensor(out, "out", _F32, dev, shape, write=True)
    lse = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if lse is None else \
        _tensor(lse, "lse", _F32, dev, shape[:-1], write=True)
    if workspace is not None:
        workspace = _tensor(workspace, "workspace", (getattr(workspace, "dtype", None),), dev,
                            getattr(workspace, "shape", None), write=True)
    s = _launch_stream(dev)
    if workspace is None:
        workspace = new_workspace(q4_workspace_size(B, T, Hq, cache._sizes[1], cache._sizes[2], max_pages), dev)
    code = lib().zf_q4_decode_attn(cache._ref, q.data_ptr(), B, T, Hq, page_table.data_ptr(), max_pages,
                                   seq_lens.data_ptr(), 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale,
                                   out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, s)
    if code:
        _check("zf_q4_decode_attn", code)
    return out, lse


@_on_stream
def q4_decode_attn_wait_test(cache: Q4Cache, q, page_table, seq_lens, scale=None, wait_limit_ns=1000000):
    """zf_q4_decode_attn_wait_test (tests of the failure path): q4_decode_attn on q [B][T][Hq][128] whose warps' first
    wait for copied records runs out after wait_limit_ns.  Returns (out, lse), which are not meaningful; the
    cache's status word gets DEV_TIMEOUT."""
    dev = cache._device
    B, T, Hq = q.shape[:3]
    q = _tensor(q, "q", _BITS16, dev, (B, T, Hq, HEAD_DIM))
    page_table, seq_lens = _tables(page_table, seq_lens, dev, B)
    max_pages = page_table.shape[1]
    s = _launch_stream(dev)
    out = torch.empty((B, T, Hq, HEAD_DIM), dtype=torch.float32, device=dev)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)
    workspace = new_workspace(q4_workspace_size(B, T, Hq, cache._sizes[1], cache._sizes[2], max_pages), dev)
    _check("zf_q4_decode_attn_wait_test",
           lib().zf_q4_decode_attn_wait_test(cache._ref, q.data_ptr(), B, T, Hq, page_table.data_ptr(), max_pages,
                                             seq_lens.data_ptr(), 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale,
                                             out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                             int(wait_limit_ns), s))
    return out, lse


def q4_chunk_workspace_size(batch, rows, num_q_heads, num_kv_heads, page_size, max_pages) -> int:
    return int(lib().zf_q4_chunk_attn_workspace_size(batch, rows, num_q_heads, num_kv_heads, page_size, max_pages))


@_on_stream
def q4_chunk_attn(cache: Q4Cache, q, page_table, seq_lens, token_start, scale=None, window=0, softcap=0.0, slopes=None,
                  out=None, lse=None, workspace=None):
    """zf_q4_chunk_attn: attention of a ragged batch of new tokens over the 4-bit cache.  q [rows][Hq][128] int16 BF16
    bits or bfloat16: rows token_start[b] .. token_start[b+1] - 1 are the last of request b's seq_lens[b] tokens
    (token_start [B+1] int32 as map_tokens gives it); page_table [>= B][*], seq_lens [>= B].  window > 0: a row
    sees that many positions, its own the last; softcap > 0: scores c tanh(s / c); slopes [Hq] float32: plus
    slopes[h] * (j - p).  Returns (out bfloat16 of q's shape, lse float32 [rows][Hq]); rows of no request are left
    as they are (undefined in tensors made here)."""
    dev = cache._device
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    shape = q.shape
    if len(shape) != 3 or shape[-1] != HEAD_DIM:
        raise ValueError(f"q: shape {list(shape)}, expected [*][*][{HEAD_DIM}]")
    q = _tensor(q, "q", _BITS16, dev, shape)
    if not isinstance(token_start, torch.Tensor) or token_start.dim() != 1 or token_start.shape[0] < 1:
        raise ValueError("token_start must be a [batch + 1] tensor")
    token_start = _tensor(token_start, "token_start", _I32, dev, token_start.shape)
    N, Hq, B = shape[0], shape[1], token_start.shape[0] - 1
    page_table, seq_lens = _tables(page_table, seq_lens, dev, B)
    max_pages = page_table.shape[1]
    slope_ptr = None
    if slopes is not None:
        slopes = _tensor(slopes, "slopes", _F32, dev, (Hq,))
        slope_ptr = slopes.data_ptr()
    out = torch.empty(shape, dtype=torch.bfloat16, device=dev) if out is None else \
        _tensor(out, "out", _BITS16, dev, shape, write=True)
    lse = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if lse is None else \
        _tensor(lse, "lse", _F32, dev, shape[:-1], write=True)
    if workspace is not None:
        workspace = _tensor(workspace, "workspace", (getattr(workspace, "dtype", None),), dev,
                            getattr(workspace, "shape", None), write=True)
    s = _launch_stream(dev)
    if workspace is None:
        workspace = new_workspace(q4_chunk_workspace_size(B, N, Hq, cache._sizes[1], cache._sizes[2], max_pages), dev)
    code = lib().zf_q4_chunk_attn(cache._ref, q.data_ptr(), N, B, Hq, token_start.data_ptr(), page_table.data_ptr(),
                                  max_pages, seq_lens.data_ptr(), 1.0 / math.sqrt(HEAD_DIM) if scale is None else scale,
                                  window, softcap, slope_ptr, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                  workspace.nbytes, s)
    if code:
        _check("zf_q4_chunk_attn", code)
    return out, lse


@_on_stream
def q4_chunk_attn_wait_test(cache: Q4Cache, q, page_table, seq_lens, token_start, wait_limit_ns=1000000):
    """zf_q4_chunk_attn_wait_test (tests of the failure path): q4_chunk_attn whose warps' first wait for work runs out
    after wait_limit_ns.  Returns (out, lse), which are not meaningful; the cache's status word gets DEV_TIMEOUT."""
    dev = cache._device
    N, Hq = q.shape[:2]
    q = _tensor(q, "q", _BITS16, dev, (N, Hq, HEAD_DIM))
    token_start = _tensor(token_start, "token_start", _I32, dev, token_start.shape)
    B = token_start.shape[0] - 1
    page_table, seq_lens = _tables(page_table, seq_lens, dev, B)
    max_pages = page_table.shape[1]
    s = _launch_stream(dev)
    out = torch.empty((N, Hq, HEAD_DIM), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    workspace = new_workspace(q4_chunk_workspace_size(B, N, Hq, cache._sizes[1], cache._sizes[2], max_pages), dev)
    _check("zf_q4_chunk_attn_wait_test",
           lib().zf_q4_chunk_attn_wait_test(cache._ref, q.data_ptr(), N, B, Hq, token_start.data_ptr(), page_table.data_ptr(),
                                            max_pages, seq_lens.data_ptr(), 1.0 / math.sqrt(HEAD_DIM), 0, 0.0, None,
                                            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                            int(wait_limit_ns), s))
    return out, lse


# ---------------------------------------------------------- slot maps and draft verification
class TokenMap(NamedTuple):
    """What zf_map_tokens gives (int32 device tensors): the requests' lengths and pages after the call, the
    position in the free list, where each request's entries start, and per new token its page, its
    index in the page and its position in the request (-1 past the last)."""
    seq_lens: torch.Tensor
    pages_held: torch.Tensor
    free_pos: torch.Tensor
    token_start: torch.Tensor
    page_ids: torch.Tensor
    positions: torch.Tensor
    seq_positions: torch.Tensor


@_on_stream
def map_tokens(page_table, seq_lens, pages_held, new_tokens, free_pages, free_pos, page_size, max_tokens, out=None,
               status=None) -> TokenMap:
    """zf_map_tokens: places for new_tokens[b] tokens of every request b, on the GPU.  page_table [B][max_pages]
    is extended in place with pages free_pages[free_pos ..]; seq_lens, pages_held, new_tokens [B], free_pages
    [F], free_pos [1], all int32 on the device.  out: a TokenMap to write into (its seq_lens, pages_held and
    free_pos may be the arguments themselves); status: an int32 device word."""
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [batch][max_pages] tensor")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a one-dimensional tensor")
    B, max_pages = page_table.shape
    dev = page_table.device
    page_table = _tensor(page_table, "page_table", _I32, dev, (B, max_pages), write=True)
    seq_lens = _tensor(seq_lens, "seq_lens", _I32, dev, (B,))
    pages_held = _tensor(pages_held, "pages_held", _I32, dev, (B,))
    new_tokens = _tensor(new_tokens, "new_tokens", _I32, dev, (B,))
    free_pages = _tensor(free_pages, "free_pages", _I32, dev, free_pages.shape)
    free_pos = _tensor(free_pos, "free_pos", _I32, dev, (1,))
    n = max(int(max_tokens), 0)
    if out is None:        # one allocation; the lists start on 16-byte boundaries
        pad = -n % 4
        if pad:
            ids, _, pos, _, seq, _, lens, held, start, free = torch.empty(
                3 * (n + pad) + 3 * B + 2, dtype=torch.int32, device=dev) \
                .unsafe_split_with_sizes((n, pad, n, pad, n, pad, B, B, B + 1, 1))
        else:
            ids, pos, seq, lens, held, start, free = torch.empty(
                3 * n + 3 * B + 2, dtype=torch.int32, device=dev).unsafe_split_with_sizes((n, n, n, B, B, B + 1, 1))
        out = TokenMap(lens, held, free, start, ids, pos, seq)
    else:
        shapes = ((B,), (B,), (1,), (B + 1,), (n,), (n,), (n,))
        out = TokenMap(*(_tensor(t, "out." + name, _I32, dev, s, write=True)
                         for t, name, s in zip(out, TokenMap._fields, shapes)))
    word = None if status is None else _tensor(status, "status", _I32, dev, (1,), write=True).data_ptr()
    s = _launch_stream(dev)
    code = lib().zf_map_tokens(B, page_size, max_pages, seq_lens.data_ptr(), pages_held.data_ptr(), new_tokens.data_ptr(),
                               page_table.data_ptr(), free_pages.data_ptr(), free_pages.shape[0], free_pos.data_ptr(),
                               out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                               out[4].data_ptr(), out[5].data_ptr(), out[6].data_ptr(), max_tokens, word, s)
    if code:
        _check("zf_map_tokens", code)
    return out


@_on_stream
def verify_drafts(target_probs, draft_tokens, uniform, draft_probs=None, n_drafts=None, seq_lens=None,
                  new_seq_lens=None, status=None, token_start=None):
    """zf_verify_drafts: target_probs [B][T+1][V] float32, draft_tokens [B][T] int32, uniform [B][T+1] float32 in
    [0, 1), draft_probs [B][T][V] float32 (None: the drafts were not sampled), n_drafts [B] int32 (None: T
    each).  Returns (accepted [B], tokens [B][T+1]) int32: the accepted drafts, one sampled token, then -1.
    With seq_lens (and new_seq_lens, which may be the same tensor) the lengths are shortened by the
    refused drafts.  token_start [B+1] int32: what map_tokens gave in this step (zf_verify_mapped_drafts); a
    request that got no places there keeps its length and gets accepted 0 and tokens -1, one that got m
    keeps m - 1 - accepted places fewer, whatever its n_drafts (at most m - 1)."""
    if not isinstance(draft_tokens, torch.Tensor) or draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be a [batch][drafts] tensor")
    B, T = draft_tokens.shape
    if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 3:
        raise ValueError("target_probs must be a [batch][drafts + 1][vocab] tensor")
    V, dev = target_probs.shape[2], draft_tokens.device
    draft_tokens = _tensor(draft_tokens, "draft_tokens", _I32, dev, (B, T))
    target_probs = _tensor(target_probs, "target_probs", _F32, dev, (B, T + 1, V))
    uniform = _tensor(uniform, "uniform", _F32, dev, (B, T + 1))
    q = n = before = after = word = None
    if draft_probs is not None:
        draft_probs = _tensor(draft_probs, "draft_probs", _F32, dev, (B, T, V))
        q = draft_probs.data_ptr()
    if n_drafts is not None:
        n_drafts = _tensor(n_drafts, "n_drafts", _I32, dev, (B,))
        n = n_drafts.data_ptr()
    if (seq_lens is None) != (new_seq_lens is None):
        raise ValueError("seq_lens and new_seq_lens go together")
    if seq_lens is not None:
        seq_lens = _tensor(seq_lens, "seq_lens", _I32, dev, (B,))
        before, after = seq_lens.data_ptr(), _tensor(new_seq_lens, "new_seq_lens", _I32, dev, (B,), write=True).data_ptr()
    if status is not None:
        word = _tensor(status, "status", _I32, dev, (1,), write=True).data_ptr()
    if token_start is not None:
        token_start = _tensor(token_start, "token_start", _I32, dev, (B + 1,))
    s = _launch_stream(dev)
    accepted = torch.empty(B, dtype=torch.int32, device=dev)
    tokens = torch.empty((B, T + 1), dtype=torch.int32, device=dev)
    if token_start is None:
        code = lib().zf_verify_drafts(B, T, V, target_probs.data_ptr(), q, draft_tokens.data_ptr(), n, uniform.data_ptr(),
                                      accepted.data_ptr(), tokens.data_ptr(), before, after, word, s)
    else:
        code = lib().zf_verify_mapped_drafts(B, T, V, target_probs.data_ptr(), q, draft_tokens.data_ptr(), n,
                                             uniform.data_ptr(), token_start.data_ptr(), accepted.data_ptr(),
                                             tokens.data_ptr(), before, after, word, s)
    if code:
        _check("zf_verify_drafts" if token_start is None else "zf_verify_mapped_drafts", code)
    return accepted, tokens


# ------------------------------------------------------------------------------------- sampling
_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@_on_stream
def sample_tokens(logits, uniform=None, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, tokens=None,
                  status=None):
    """zf_sample_tokens: logits [R][V] float32, bfloat16 or float16 (rows may be a stride apart); uniform [R] float32 in
    [0, 1); temperature, top_p, min_p [R] float32 and top_k [R] int32, each None for none (min_p: 0 or less too).
    Returns tokens [R] int32 (None when uniform is None).  probs [R][V] float32 is filled with the distribution sampled from; uniform may be
    None when only that is wanted.  tokens: a tensor to write into; status: an int32 device word."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [rows][vocab] tensor")
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits: dtype {logits.dtype}, expected torch.float32, torch.bfloat16 or torch.float16")
    R, V = logits.shape
    dev = logits.device
    if logits.stride(1) != 1 or logits.stride(0) < V:
        logits = logits.contiguous()
    rows = (R,)
    u = t = k = p = m = out = dist = word = None
    if uniform is not None:
        u = (uniform := _tensor(uniform, "uniform", _F32, dev, rows)).data_ptr()
    elif tokens is not None:
        raise ValueError("tokens need uniform")
    elif probs is None:
        raise ValueError("uniform, probs or both are needed")
    if temperature is not None:
        t = (temperature := _tensor(temperature, "temperature", _F32, dev, rows)).data_ptr()
    if top_k is not None:
        k = (top_k := _tensor(top_k, "top_k", _I32, dev, rows)).data_ptr()
    if top_p is not None:
        p = (top_p := _tensor(top_p, "top_p", _F32, dev, rows)).data_ptr()
    if min_p is not None:
        m = (min_p := _tensor(min_p, "min_p", _F32, dev, rows)).data_ptr()
    if probs is not None:
        dist = _tensor(probs, "probs", _F32, dev, (R, V), write=True).data_ptr()
    if status is not None:
        word = _tensor(status, "status", _I32, dev, (1,), write=True).data_ptr()
    s = _launch_stream(dev)
    if uniform is not None:
        tokens = torch.empty(R, dtype=torch.int32, device=dev) if tokens is None else \
            _tensor(tokens, "tokens", _I32, dev, rows, write=True)
        out = tokens.data_ptr()
    code = lib().zf_sample_tokens(R, V, logits.data_ptr(), kind, max(logits.stride(0), V), u, t, k, p, m, out, dist, word, s)
    if code:
        _check("zf_sample_tokens", code)
    return tokens


# ------------------------------------------------------------ sharing, freeing and moving pages
class Fork(NamedTuple):
    """What zf_fork_requests gives: the requests' lengths and pages after the call, the position in the free list, and
    per entry the page to copy and where to (-1: none)."""
    seq_lens: torch.Tensor
    pages_held: torch.Tensor
    free_pos: torch.Tensor
    copy_src: torch.Tensor
    copy_dst: torch.Tensor


class Release(NamedTuple):
    """What zf_release_requests gives: lengths and pages after the call, and the position in the free list."""
    seq_lens: torch.Tensor
    pages_held: torch.Tensor
    free_pos: torch.Tensor


class Compaction(NamedTuple):
    """What zf_compact_pages gives: the renumbered page table, a free list over the whole pool and the position in it
    (the number of pages in use), and the pages to copy and where to (-1 past the last)."""
    page_table: torch.Tensor
    free_pages: torch.Tensor
    free_pos: torch.Tensor
    copy_src: torch.Tensor
    copy_dst: torch.Tensor


def _table_2d(page_table):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [batch][max_pages] tensor")
    return page_table.shape


def _list_1d(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name} must be a one-dimensional tensor")
    return t.shape


def _outputs(kind, out, sizes, dev):
    """The one-dimensional int32 outputs of a call as `kind`: made here (in one allocation), or `out` checked."""
    if out is not None:
        return kind(*[_tensor(t, "out." + name, _I32, dev, (n,), write=True) for t, name, n in zip(out, kind._fields, sizes)])
    return kind._make(torch.empty(sum(sizes), dtype=torch.int32, device=dev).unsafe_split_with_sizes(sizes))


def _status_ptr(status, dev):
    return None if status is None else _tensor(status, "status", _I32, dev, (1,), write=True).data_ptr()


def _workspace(workspace, nbytes, dev):
    if workspace is None:
        return new_workspace(nbytes, dev)
    return _tensor(workspace, "workspace", (getattr(workspace, "dtype", None),), dev, getattr(workspace, "shape", None),
                   write=True)


@_on_stream
def fork_requests(page_table, seq_lens, pages_held, src, dst, free_pages, free_pos, page_size, out=None, status=None) -> Fork:
    """zf_fork_requests: rows dst[i] of page_table [B][max_pages] (empty ones) go on from rows src[i]: full pages are
    shared, a last page that is not full gets a page from free_pages[free_pos ..].  seq_lens, pages_held [B], src,
    dst [n], free_pages [F], free_pos [1], all int32 on the device; page_table is written in place.  Then, per layer:
    q4_copy_pages(cache, fork.copy_src, fork.copy_dst).  out: a Fork to write into (its seq_lens, pages_held and
    free_pos may be the arguments themselves); status: an int32 device word."""
    B, max_pages = _table_2d(page_table)
    dev = page_table.device
    page_table = _tensor(page_table, "page_table", _I32, dev, (B, max_pages), write=True)
    seq_lens = _tensor(seq_lens, "seq_lens", _I32, dev, (B,))
    pages_held = _tensor(pages_held, "pages_held", _I32, dev, (B,))
    src = _tensor(src, "src", _I32, dev, _list_1d(src, "src"))
    n = src.shape[0]
    dst = _tensor(dst, "dst", _I32, dev, (n,))
    free_pages = _tensor(free_pages, "free_pages", _I32, dev, _list_1d(free_pages, "free_pages"))
    free_pos = _tensor(free_pos, "free_pos", _I32, dev, (1,))
    word = _status_ptr(status, dev)
    s = _launch_stream(dev)
    out = _outputs(Fork, out, (B, B, 1, n, n), dev)
    code = lib().zf_fork_requests(B, page_size, max_pages, seq_lens.data_ptr(), pages_held.data_ptr(), src.data_ptr(),
                                  dst.data_ptr(), n, page_table.data_ptr(), free_pages.data_ptr(), free_pages.shape[0],
                                  free_pos.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(),
                                  out[3].data_ptr(), out[4].data_ptr(), word, s)
    if code:
        _check("zf_fork_requests", code)
    return out


@_on_stream
def q4_copy_pages(cache: Q4Cache, src, dst):
    """zf_q4_copy_pages: pages src[i] to dst[i], int32 on the device (both -1: skipped); no page may be a destination
    twice, nor a source and a destination."""
    src = _tensor(src, "src", _I32, cache._device, _list_1d(src, "src"))
    dst = _tensor(dst, "dst", _I32, cache._device, src.shape)
    s = _launch_stream(cache._device)
    code = lib().zf_q4_copy_pages(cache._ref, src.data_ptr(), dst.data_ptr(), src.shape[0], s)
    if code:
        _check("zf_q4_copy_pages", code)


@_on_stream
def release_requests(page_table, seq_lens, pages_held, release, free_pages, free_pos, num_pages, out=None, status=None,
                     workspace=None) -> Release:
    """zf_release_requests: the rows with release[b] != 0 give back the pages that no other row holds, into
    free_pages[.. free_pos - 1] (written in place).  page_table [B][max_pages], seq_lens, pages_held, release [B],
    free_pages [F], free_pos [1], all int32 on the device.  out: a Release to write into (its tensors may be the
    arguments); status: an int32 device word; workspace: see release_workspace_size."""
    B, max_pages = _table_2d(page_table)
    dev = page_table.device
    page_table = _tensor(page_table, "page_table", _I32, dev, (B, max_pages))
    seq_lens = _tensor(seq_lens, "seq_lens", _I32, dev, (B,))
    pages_held = _tensor(pages_held, "pages_held", _I32, dev, (B,))
    release = _tensor(release, "release", _I32, dev, (B,))
    free_pages = _tensor(free_pages, "free_pages", _I32, dev, _list_1d(free_pages, "free_pages"), write=True)
    free_pos = _tensor(free_pos, "free_pos", _I32, dev, (1,))
    word = _status_ptr(status, dev)
    s = _launch_stream(dev)
    out = _outputs(Release, out, (B, B, 1), dev)
    workspace = _workspace(workspace, release_workspace_size(num_pages), dev)
    code = lib().zf_release_requests(B, max_pages, num_pages, page_table.data_ptr(), seq_lens.data_ptr(),
                                     pages_held.data_ptr(), release.data_ptr(), free_pages.data_ptr(),
                                     free_pages.shape[0], free_pos.data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                                     out[2].data_ptr(), word, workspace.data_ptr(), workspace.nbytes, s)
    if code:
        _check("zf_release_requests", code)
    return out


@_on_stream
def compact_pages(page_table, pages_held, num_pages, out=None, status=None, workspace=None) -> Compaction:
    """zf_compact_pages: the pages in use, n of them, get the ids 0 .. n - 1.  page_table [B][max_pages], pages_held
    [B], int32 on the device.  Then, per layer: q4_copy_pages(cache, c.copy_src, c.copy_dst).  out: a Compaction to
    write into (its page_table may be the argument); status: an int32 device word; workspace: see
    compact_workspace_size."""
    B, max_pages = _table_2d(page_table)
    dev = page_table.device
    page_table = _tensor(page_table, "page_table", _I32, dev, (B, max_pages))
    pages_held = _tensor(pages_held, "pages_held", _I32, dev, (B,))
    if num_pages < 0:
        raise ValueError("num_pages must not be negative")
    word = _status_ptr(status, dev)
    s = _launch_stream(dev)
    sizes = (B * max_pages, num_pages, 1, num_pages // 2, num_pages // 2)
    if out is None:
        table, *lists = torch.empty(sum(sizes), dtype=torch.int32, device=dev).unsafe_split_with_sizes(sizes)
        out = Compaction(table.view(B, max_pages), *lists)
    else:
        out = Compaction(*[_tensor(t, "out." + name, _I32, dev, (n,) if i else (B, max_pages), write=True)
                           for i, (t, name, n) in enumerate(zip(out, Compaction._fields, sizes))])
    workspace = _workspace(workspace, compact_workspace_size(num_pages), dev)
    code = lib().zf_compact_pages(B, max_pages, num_pages, page_table.data_ptr(), pages_held.data_ptr(), out[0].data_ptr(),
                                  out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), word,
                                  workspace.data_ptr(), workspace.nbytes, s)
    if code:
        _check("zf_compact_pages", code)
    return out


def release_workspace_size(num_pages) -> int:
    return int(lib().zf_release_requests_workspace_size(num_pages))


def compact_workspace_size(num_pages) -> int:
    return int(lib().zf_compact_pages_workspace_size(num_pages))


# --------------------------------------------------------------------------------- page manager
ERR_CAPACITY = -6


def _i32(values):
    arr = (_c_int32 * max(len(values), 1))(*values)
    return arr


class KvManager:
    """zf_kv: host-side page manager (page ids for all layers, one raw-slot pool shared by
    num_layers layers).  admit/append return the write list (page_ids, n_valid, raw_slots) with
    raw_slots[l] the slot list of layer l's call: encode_pages for a prompt, append_tokens
    (positions n_valid - 1) for a decode step."""

    def __init__(self, num_pages, num_raw_slots, page_size, max_requests, max_pages_per_req, num_layers=1):
        self.page_size, self.max_requests, self.max_pages = page_size, max_requests, max_pages_per_req
        self.num_layers = num_layers
        h = _c_void_p()
        _check("zf_kv_create", lib().zf_kv_create(num_pages, num_raw_slots, num_layers, page_size, max_requests,
                                                   max_pages_per_req, ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            lib().zf_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _layers(self, flat, n):
        return [list(flat[l * n:(l + 1) * n]) for l in range(self.num_layers)]

    def admit(self, req, length):
        n_max = max(-(-length // self.page_size), 1)
        ids, nv, n = (_c_int32 * n_max)(), (_c_int32 * n_max)(), _c_int32()
        rs = (_c_int32 * (n_max * self.num_layers))()
        _check("zf_kv_admit", lib().zf_kv_admit(self._h, req, length, ids, nv, rs, ctypes.byref(n)))
        k = n.value
        return list(ids[:k]), list(nv[:k]), self._layers(rs, k)

    def append(self, reqs):
        n = len(reqs)
        ids, nv = (_c_int32 * max(n, 1))(), (_c_int32 * max(n, 1))()
        rs = (_c_int32 * max(n * self.num_layers, 1))()
        _check("zf_kv_append", lib().zf_kv_append(self._h, _i32(reqs), n, ids, nv, rs))
        return list(ids[:n]), list(nv[:n]), self._layers(rs, n)

    def pending(self):
        """(page ids, raw slots per layer) of the full pages awaiting reclaim, ascending id."""
        n = _c_int32()
        code = lib().zf_kv_pending(self._h, None, None, 0, ctypes.byref(n))
        if code not in (0, -1):
            _check("zf_kv_pending", code)
        k = n.value
        ids, rs = (_c_int32 * max(k, 1))(), (_c_int32 * max(k * self.num_layers, 1))()
        _check("zf_kv_pending", lib().zf_kv_pending(self._h, ids, rs, k, ctypes.byref(n)))
        return list(ids[:k]), self._layers(rs, k)

    def reclaim(self, page_ids, kept_raw):
        """kept_raw[l][i]: page_ids[i] has a page-head stored raw in layer l (keeps that layer's slot)."""
        n = len(page_ids)
        if len(kept_raw) != self.num_layers or any(len(row) != n for row in kept_raw):
            raise ValueError("kept_raw needs one row of len(page_ids) flags per layer")
        flat = [int(bool(x)) for row in kept_raw for x in row]
        _check("zf_kv_reclaim", lib().zf_kv_reclaim(self._h, _i32(page_ids), _i32(flat), n))

    def reclaim_from(self, caches):
        """Reclaim every pending page from the directories of `caches`.  With num_layers layers,
        caches[l] is layer l (each layer keeps or returns its own slot); with num_layers == 1, any
        number of caches addressed by the same slots (a page keeps its slot if it is raw in any)."""
        ids, _ = self.pending()
        if not ids:
            return 0
        if self.num_layers > 1 and len(caches) != self.num_layers:
            raise ValueError("one cache per layer")
        idx = torch.as_tensor(ids, dtype=torch.long)
        raw = [(c.dir.index_select(0, idx.to(c.dir.device)).cpu() >= 0).any(dim=1) for c in caches]
        if self.num_layers == 1:
            kept = [torch.stack(raw).any(dim=0).tolist()]
        else:
            kept = [r.tolist() for r in raw]
        self.reclaim(ids, kept)
        return len(ids)

    def release(self, req):
        _check("zf_kv_release", lib().zf_kv_release(self._h, req))

    def export(self):
        """(page_table [max_requests][max_pages_per_req], seq_lens [max_requests]) int32 CPU tensors."""
        table = torch.empty((self.max_requests, self.max_pages), dtype=torch.int32)
        lens = torch.empty(self.max_requests, dtype=torch.int32)
        _check("zf_kv_export", lib().zf_kv_export(self._h, ctypes.cast(table.data_ptr(), _P32),
                                                   ctypes.cast(lens.data_ptr(), _P32)))
        return table, lens

    def stats(self) -> dict:
        st = ZfKvStats()
        _check("zf_kv_get_stats", lib().zf_kv_get_stats(self._h, ctypes.byref(st)))
        return {name: getattr(st, name) for name, _ in ZfKvStats._fields_}


def kv_plan_pages(bytes_per_layer, num_kv_heads, page_size, num_raw_slots):
    """(page ids, dense pages) that bytes_per_layer holds (zf_kv_plan_pages)."""
    a, b = _c_int32(), _c_int32()
    _check("zf_kv_plan_pages", lib().zf_kv_plan_pages(int(bytes_per_layer), num_kv_heads, page_size, num_raw_slots,
                                                       ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value
