"""Python binding of the attention entry points next to the indexer.

Argument marshalling only, with the checks that need a tensor (type, shape,
layout, device); lengths, heads and page geometry are checked by the library.
The arguments and results are those of include/dosa_indexer.h:

    dsa_prompt_attention   causal attention of packed sequences
    Cache                  a paged cache of keys and values in 4 bits
    dsa_cache_append/read  quantise tokens into it, read them back
    dsa_cache_attention    attention over it, every key or the selected ones
    dsa_cache_weights      attention weight each cached key received
    dsa_cache_evict        keep the keys that received most

Calls run on ``stream`` (a torch stream of the tensors' device or a handle of
one; default: its current stream) and raise :class:`DosaError`.  ``workspace``
is a device tensor of at least the matching ``*_workspace_size`` bytes.
"""
from __future__ import annotations

import array
import ctypes
from typing import Optional, Sequence

_I32, _I64, _F32, _VP, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class DsaCache(ctypes.Structure):
    _fields_ = [("k_codes", _VP), ("k_scales", _VP), ("v_codes", _VP), ("v_scales", _VP), ("page_table", _VP),
                ("num_pages", _I32), ("page_size", _I32), ("max_pages", _I32), ("Hkv", _I32), ("d", _I32),
                ("reserved", _I32)]


class DsaEvictArray(ctypes.Structure):
    _fields_ = [("src", _VP), ("dst", _VP), ("row_bytes", _I64)]


def declare(L) -> None:
    """Argument types of the attention entry points of a loaded library."""
    pc = ctypes.POINTER(DsaCache)
    for name, args, res in (
        ("dsa_prompt_workspace_size", [_I32, _VP, _VP, _I32, _I32, _I32, _I32], _SZ),
        ("dsa_prompt_attention", [_VP, _I64, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _F32, _VP,
                                  _VP, _VP, _SZ, _VP], ctypes.c_int),
        ("dsa_cache_append", [pc, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _I32, _VP, _VP, _VP], ctypes.c_int),
        ("dsa_cache_read", [pc, _VP, _I64, _VP, _I64, _I32, _VP, _VP, _I32, _VP], ctypes.c_int),
        ("dsa_cache_workspace_size", [_I32, _VP, _VP, _I32, _I32, _I32, _I32], _SZ),
        ("dsa_cache_attention", [pc, _VP, _I64, _I32, _VP, _VP, _I32, _I32, _VP, _I32, _F32, _VP, _VP, _VP, _SZ, _VP],
         ctypes.c_int),
        ("dsa_weights_workspace_size", [_I32, _VP, _VP, _I32, _I32, _I32], _SZ),
        ("dsa_cache_weights", [pc, _VP, _I64, _I32, _VP, _VP, _VP, _I32, _I32, _F32, _VP, _VP, _VP, _SZ, _VP],
         ctypes.c_int),
        ("dsa_evict_workspace_size", [_I32, _VP, _VP], _SZ),
        ("dsa_cache_evict", [_VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP, _I32, _I32, _I32, _VP, _I32, _VP, _I32,
                             _VP, _SZ, _VP], ctypes.c_int),
    ):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


_loaded = _torch = _device = _stream = None


def _lib():
    global _loaded, _torch, _device, _stream
    if _loaded is None:
        import torch

        from . import lib

        _loaded, _torch = lib(), torch
        # the current device, and the handle of torch.cuda.current_stream(): without the objects where torch has
        # such functions (they are not among its public ones)
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _loaded


def _bad(msg: str):
    from . import DosaError

    raise DosaError(-1, msg)


def _check(st: int) -> None:
    if st != 0:
        from . import DosaError, status_string

        raise DosaError(st, status_string(st))


class _lens:
    """Host lengths as an argument of the library; ctypes keeps the object, and so the array, for the call."""

    __slots__ = ("data", "_as_parameter_")

    def __init__(self, v: Sequence[int]):
        try:
            self.data = array.array("i", v) if len(v) else array.array("i", (0,))
        except (TypeError, OverflowError):
            _bad("lengths must be integers below 2^31")
        self._as_parameter_ = self.data.buffer_info()[0]


_codes = {"f32": 0, "bf16": 1}


def _code(dtype, what: str) -> int:
    code = _codes.get(dtype)
    if code is None:
        code = {"torch.float32": 0, "torch.bfloat16": 1}.get(str(dtype))
        if code is None:
            _bad(f"{what}: type {dtype} (float32 and bfloat16 are supported)")
        _codes[dtype] = code
    return code


def _size(n: int, what: str) -> int:
    if n == 0:
        from . import DosaError

        raise DosaError(-2, f"{what}: invalid or unsupported lengths or heads")
    return int(n)


def _rows(t, name: str, heads: int, d: int, tokens: int, like, contiguous: bool = False) -> int:
    """Token stride of a packed operand [tokens, heads, d] of `like`'s type and device."""
    if t.shape != (tokens, heads, d):
        _bad(f"{name} must be [{tokens}, {heads}, {d}], is {list(t.shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        _bad(f"{name} must be {like.dtype} on {like.device}, is {t.dtype} on {t.device}")
    if tokens == 0:
        return heads * d
    s = t.stride()
    if (s[2] != 1 and d > 1) or (heads > 1 and s[1] != d):
        _bad(f"{name}: the heads of a token must lie together")
    if tokens == 1:
        return heads * d
    if contiguous and s[0] != heads * d:
        _bad(f"{name} must be contiguous")
    return s[0]


def _tensor(t, name: str, dtype, shape, device) -> Optional[int]:
    """Address of a contiguous tensor of the given type, shape and device."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        _bad(f"{name} must be a contiguous {dtype} {list(shape)} on {device}, is {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _space(ws, device):
    if ws is None:
        return None, 0
    if not ws.is_contiguous() or ws.device != device:
        _bad(f"workspace must be contiguous and on {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


class _On:
    """The stream to run on, with the tensors' device current."""

    __slots__ = ("back", "device", "stream")

    def __init__(self, device, stream):
        self.device, self.stream, self.back = device, stream, None

    def __enter__(self) -> int:
        torch = _torch
        if self.device.type != "cuda":
            _bad(f"tensors are on {self.device}, not on a GPU")
        if getattr(self.stream, "device", self.device) != self.device:
            _bad(f"stream is of {self.stream.device}, the tensors are on {self.device}")
        if _device() != self.device.index:
            self.back = torch.cuda.device(self.device)
            self.back.__enter__()
        if self.stream is None:
            return _stream(self.device.index)
        return int(getattr(self.stream, "cuda_stream", self.stream))

    def __exit__(self, *exc):
        if self.back is not None:
            self.back.__exit__(*exc)


_on = _On


class Cache:
    """A paged cache of keys and values in 4 bits.

    k_codes, v_codes uint8 [num_pages, page_size, Hkv, d/2], k_scales, v_scales
    uint8 [num_pages, page_size, Hkv, d/32], page_table int32 [batch,
    max_pages], all contiguous on one device.  :meth:`empty` allocates one.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, page_table):
        import torch

        if k_codes.dim() != 4 or k_codes.dtype != torch.uint8:
            _bad("k_codes must be uint8 [num_pages, page_size, Hkv, d/2]")
        pages, page, heads, half = k_codes.shape
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.page_table = page_table
        self.num_pages, self.page_size, self.Hkv, self.d = pages, page, heads, 2 * half
        self.device = k_codes.device
        for name, w in (("k_codes", half), ("k_scales", half // 16), ("v_codes", half), ("v_scales", half // 16)):
            _tensor(getattr(self, name), name, torch.uint8, (pages, page, heads, w), self.device)
        if page_table.dim() != 2:
            _bad("page_table must be int32 [batch, max_pages]")
        _tensor(page_table, "page_table", torch.int32, page_table.shape, self.device)
        self.batch, self.max_pages = page_table.shape
        self.struct = DsaCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                               page_table.data_ptr(), pages, page, self.max_pages, heads, 2 * half, 0)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, Hkv: int, d: int, page_table):
        import torch

        mk = lambda w: torch.empty(num_pages, page_size, Hkv, w, dtype=torch.uint8, device=page_table.device)
        return cls(mk(d // 2), mk(d // 32), mk(d // 2), mk(d // 32), page_table)

    def _batch(self, q_lens, kv_lens) -> int:
        if not (len(q_lens) == len(kv_lens) <= self.batch):
            _bad(f"{len(q_lens)} q_lens, {len(kv_lens)} kv_lens for a page table of {self.batch} rows")
        return len(q_lens)

    def arrays(self):
        """(src, dst) pairs of the cache's buffers for :func:`dsa_cache_evict`, in place."""
        return [(t, t) for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales)]


def prompt_workspace_size(q_lens, kv_lens, Hq: int, Hkv: int, d: int, dtype) -> int:
    return _size(_lib().dsa_prompt_workspace_size(len(q_lens), _lens(q_lens), _lens(kv_lens), Hq, Hkv, d,
                                                  _code(dtype, "dtype")), "prompt attention")


def dsa_prompt_attention(q, k, v, q_lens, kv_lens, out, lse=None, scale: Optional[float] = None, workspace=None,
                         stream=None):
    """Causal attention of packed sequences: q, out [total_q, Hq, d], k, v [total_k, Hkv, d], lse
    [total_q, Hq] fp32 or None; scale defaults to d ** -0.5."""
    L, torch = _lib(), _torch
    if q.dim() != 3 or k.dim() != 3:
        _bad("q and k must be [tokens, heads, d]")
    if len(q_lens) != len(kv_lens):
        _bad("q_lens and kv_lens differ in length")
    (_, hq, d), hk = q.shape, k.shape[1]
    nq, nk = sum(q_lens), sum(kv_lens)
    sq, sk, sv = _rows(q, "q", hq, d, nq, q), _rows(k, "k", hk, d, nk, q), _rows(v, "v", hk, d, nk, q)
    _rows(out, "out", hq, d, nq, q, True)
    plse = _tensor(lse, "lse", torch.float32, (nq, hq), q.device)
    ws, n = _space(workspace, q.device)
    with _on(q.device, stream) as st:
        _check(L.dsa_prompt_attention(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, _code(q.dtype, "q"),
                                           _lens(q_lens), _lens(kv_lens), len(q_lens), hq, hk, d,
                                           d ** -0.5 if scale is None else scale, out.data_ptr(), plse, ws, n, st))


def _io(fn, cache, k, v, q_lens, kv_lens, extra, stream):
    n = cache._batch(q_lens, kv_lens)
    if k.device != cache.device:
        _bad(f"k must be on {cache.device}")
    nq = sum(q_lens)
    sk, sv = _rows(k, "k", cache.Hkv, cache.d, nq, k), _rows(v, "v", cache.Hkv, cache.d, nq, k)
    with _on(k.device, stream) as st:
        _check(fn(ctypes.byref(cache.struct), k.data_ptr(), sk, v.data_ptr(), sv, _code(k.dtype, "k"), _lens(q_lens),
                  _lens(kv_lens), n, *extra, st))


def dsa_cache_append(cache: Cache, k, v, q_lens, kv_lens, pos=None, seen_lens=None, stream=None):
    """Quantise the newest q_lens[b] tokens of each sequence, k, v [total_q, Hkv, d], into the cache; pos
    int32 [num_pages, page_size] gets their places in the text."""
    L, torch = _lib(), _torch
    p = _tensor(pos, "pos", torch.int32, (cache.num_pages, cache.page_size), cache.device)
    if seen_lens is not None and len(seen_lens) != len(kv_lens):
        _bad("seen_lens and kv_lens differ in length")
    _io(L.dsa_cache_append, cache, k, v, q_lens, kv_lens, (p, None if seen_lens is None else _lens(seen_lens)), stream)


def dsa_cache_read(cache: Cache, k, v, q_lens, kv_lens, stream=None):
    """Read the newest q_lens[b] tokens of each sequence back into k, v [total_q, Hkv, d]."""
    _io(_lib().dsa_cache_read, cache, k, v, q_lens, kv_lens, (), stream)


def cache_workspace_size(q_lens, kv_lens, Hq: int, Hkv: int, d: int, topk: int = 0) -> int:
    return _size(_lib().dsa_cache_workspace_size(len(q_lens), _lens(q_lens), _lens(kv_lens), Hq, Hkv, d, topk),
                 "cache attention")


def dsa_cache_attention(cache: Cache, q, q_lens, kv_lens, out, lse=None, idx=None, scale: Optional[float] = None,
                        workspace=None, stream=None):
    """Attention over the cache: q, out [total_q, Hq, d]; idx int32 [total_q, topk] restricts each query
    to the keys it lists (an indexer's out_idx)."""
    L, torch = _lib(), _torch
    n = cache._batch(q_lens, kv_lens)
    nq = sum(q_lens)
    if q.dim() != 3 or q.device != cache.device:
        _bad(f"q must be [tokens, heads, d] on {cache.device}")
    hq = q.shape[1]
    sq = _rows(q, "q", hq, cache.d, nq, q)
    _rows(out, "out", hq, cache.d, nq, q, True)
    plse = _tensor(lse, "lse", torch.float32, (nq, hq), q.device)
    topk = 0
    if idx is not None:
        if idx.dim() != 2 or idx.shape[1] == 0:
            _bad("idx must be int32 [total_q, topk], topk at least 1")
        topk = idx.shape[1]
    pidx = _tensor(idx, "idx", torch.int32, (nq, topk), q.device)
    if idx is not None and nq == 0:
        return
    ws, nb = _space(workspace, q.device)
    with _on(q.device, stream) as st:
        _check(L.dsa_cache_attention(ctypes.byref(cache.struct), q.data_ptr(), sq, _code(q.dtype, "q"),
                                          _lens(q_lens), _lens(kv_lens), n, hq, pidx, topk,
                                          cache.d ** -0.5 if scale is None else scale, out.data_ptr(), plse, ws, nb, st))


def weights_workspace_size(q_lens, kv_lens, Hq: int, Hkv: int, d: int) -> int:
    return _size(_lib().dsa_weights_workspace_size(len(q_lens), _lens(q_lens), _lens(kv_lens), Hq, Hkv, d),
                 "cache weights")


def dsa_cache_weights(cache: Cache, q, lse, q_lens, kv_lens, acc, acc_out, scale: Optional[float] = None,
                      workspace=None, stream=None):
    """acc_out = acc (0 for the call's own tokens; None: 0) + the weight each key received from the
    queries whose normalisers are lse; acc, acc_out fp32 [num_pages, page_size]."""
    L, torch = _lib(), _torch
    n = cache._batch(q_lens, kv_lens)
    nq = sum(q_lens)
    if q.dim() != 3 or q.device != cache.device:
        _bad(f"q must be [tokens, heads, d] on {cache.device}")
    hq = q.shape[1]
    sq = _rows(q, "q", hq, cache.d, nq, q)
    plse = _tensor(lse, "lse", torch.float32, (nq, hq), q.device)
    shape = (cache.num_pages, cache.page_size)
    pa = _tensor(acc, "acc", torch.float32, shape, q.device)
    po = _tensor(acc_out, "acc_out", torch.float32, shape, q.device)
    ws, nb = _space(workspace, q.device)
    with _on(q.device, stream) as st:
        _check(L.dsa_cache_weights(ctypes.byref(cache.struct), q.data_ptr(), sq, _code(q.dtype, "q"), plse,
                                        _lens(q_lens), _lens(kv_lens), n, hq,
                                        cache.d ** -0.5 if scale is None else scale, pa, po, ws, nb, st))


def evict_workspace_size(kv_lens, new_lens) -> int:
    return _size(_lib().dsa_evict_workspace_size(len(kv_lens), _lens(kv_lens), _lens(new_lens)), "eviction")


def dsa_cache_evict(acc, page_table, kv_lens, new_lens, arrays, out_src, pos=None, seen_lens=None, prefix: int = 0,
                    window: int = 0, workspace=None, stream=None):
    """Keep the new_lens[b] keys of largest acc of each sequence and move the rows of ``arrays``, (src, dst)
    pairs of contiguous tensors [num_pages, page_size, ...] (dst may be src); out_src int32 [batch, >= new_len]
    gets the index each kept key came from."""
    L, torch = _lib(), _torch
    if acc.dim() != 2 or page_table.dim() != 2 or out_src.dim() != 2:
        _bad("acc must be [num_pages, page_size], page_table [batch, max_pages], out_src [batch, n]")
    n = len(kv_lens)
    if len(new_lens) != n or page_table.shape[0] < n or out_src.shape[0] < n or \
            (seen_lens is not None and len(seen_lens) != n):
        _bad("kv_lens, new_lens, seen_lens, page_table and out_src differ in length")
    dev = acc.device
    pacc = _tensor(acc, "acc", torch.float32, acc.shape, dev)
    ptab = _tensor(page_table, "page_table", torch.int32, page_table.shape, dev)
    ppos = _tensor(pos, "pos", torch.int32, acc.shape, dev)
    psrc = _tensor(out_src, "out_src", torch.int32, out_src.shape, dev)
    recs = (DsaEvictArray * max(len(arrays), 1))()
    for i, (a, b) in enumerate(arrays):
        for t in (a, b):
            if tuple(t.shape[:2]) != tuple(acc.shape) or not t.is_contiguous() or t.device != dev:
                _bad(f"array {i} must be contiguous [{acc.shape[0]}, {acc.shape[1]}, ...] on {dev}")
        if a.shape != b.shape or a.dtype != b.dtype:
            _bad(f"array {i}: src and dst differ")
        recs[i] = DsaEvictArray(a.data_ptr(), b.data_ptr(), a[0, 0].numel() * a.element_size() if a.numel() else 0)
    ws, nb = _space(workspace, dev)
    with _on(dev, stream) as st:
        _check(L.dsa_cache_evict(pacc, ppos, ptab, acc.shape[1], page_table.shape[1], acc.shape[0], _lens(kv_lens),
                                      _lens(new_lens), None if seen_lens is None else _lens(seen_lens), n, prefix, window,
                                      recs, len(arrays), psrc, out_src.shape[1], ws, nb, st))
